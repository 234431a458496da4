// Writing the quantised KV cache and reading it back.
//
// A cache row is one token of one KV head.  The write maps its D bf16 values x to one fp32 scale
// and D codes ("Flash Attention on Ascend: three techniques", section 3, KV compression):
//   scale = fl32(max|x| / m)       code = clamp(rint(fl32(x / scale)), -m, m)       m = 127 or 7
// with ties to even and code 0 where the scale is 0; a row that holds an infinity or a NaN gets
// scale NaN and codes 0, so that whatever reads it is NaN rather than silently wrong.  The read
// is bf16(fl32(code * scale)).  Both move every byte once and are bound by HBM.
//
// Both kernels see the cache as pages of P tokens: codes [page][P][Hkv][row bytes], scales
// [page][Hkv][P].  A contiguous cache [B, S, Hkv, ...] is the case P = S, page = sequence.
//
// Layout of the work: one warp takes 32 consecutive tokens of one KV head, of K or of V, so that
// the 32 scales (consecutive in memory) move as one coalesced access, lane = token.  A row is
// spread over D / 16 lanes, each with two 8-value chunks D / 2 apart, so every access of a row is
// contiguous over its lanes; consecutive warps of a block take consecutive heads, which
// are adjacent in memory.
#pragma once

#include "sm100.cuh"

namespace fa {

// Where the tokens of a call live in the cache.
struct KvMap {
  const int32_t* cu_tokens;    // [B + 1] first token of each sequence, or null: per_seq each
  const int32_t* positions;    // [B] position of each sequence's first token, or null: 0
  const int32_t* block_table;  // [B, max_pages]; null: contiguous cache, page = sequence
  int N;                       // tokens
  int B, per_seq, Hkv;
  int page_size, page_shift, max_pages, num_pages;
};

struct KvCopyParams {
  KvMap map;
  const uint16_t *k, *v;  // bf16 token rows [N][Hkv][D] (source of the write)
  uint16_t *k_out, *v_out;  // ... (destination of the read)
  long long k_stride, v_stride;  // elements between token rows
  uint8_t *k_codes, *v_codes;
  float *k_scale, *v_scale;
};

// Page and row of token i (page < 0: not covered by any sequence, or an index out of range,
// which is recorded in the status word).
template <bool kPaged>
__device__ __forceinline__ void kv_locate(const KvMap& m, int i, int& page, int& row) {
  page = -1;
  row = 0;
  if (i >= m.N) return;
  if constexpr (!kPaged) {
    page = i / m.per_seq;
    row = i - page * m.per_seq;
  } else {
    int b, first;
    if (m.cu_tokens != nullptr) {
      if (i >= m.cu_tokens[m.B]) return;  // behind the last sequence
      // the last sequence that starts at or before token i (empty ones start where the next does)
      int lo = 0, hi = m.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (m.cu_tokens[mid] <= i) lo = mid; else hi = mid;
      }
      b = lo;
      first = m.cu_tokens[lo];
      if (first > i || m.cu_tokens[lo + 1] <= i) {  // not ascending from 0
        atomicOr(&g_fa_device_status, kDevStatusBadIndex);
        return;
      }
    } else {
      b = i / m.per_seq;
      first = b * m.per_seq;
    }
    const long long pos =
        (m.positions != nullptr ? static_cast<long long>(m.positions[b]) : 0) + (i - first);
    if (pos < 0 || pos >= (static_cast<long long>(m.max_pages) << m.page_shift)) {
      atomicOr(&g_fa_device_status, kDevStatusBadIndex);
      return;
    }
    const int pg = m.block_table[static_cast<size_t>(b) * m.max_pages + (pos >> m.page_shift)];
    if (static_cast<unsigned>(pg) >= static_cast<unsigned>(m.num_pages)) {
      atomicOr(&g_fa_device_status, kDevStatusBadIndex);
      return;
    }
    page = pg;
    row = static_cast<int>(pos) & (m.page_size - 1);
  }
}

// The first block reports token offsets that do not start at 0, do not ascend, or pass N.
__device__ __forceinline__ void kv_check_cu(const KvMap& m) {
  if (m.cu_tokens == nullptr || blockIdx.x != 0) return;
  bool bad = false;
  for (int b = threadIdx.x; b <= m.B; b += blockDim.x) {
    const int c = m.cu_tokens[b];
    bad |= c < 0 || c > m.N || (b == 0 ? c != 0 : c < m.cu_tokens[b - 1]);
  }
  if (bad) atomicOr(&g_fa_device_status, kDevStatusBadIndex);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// Codes of the 8 bf16 values in x, one per low byte (two's complement) of c.  `exact`: every
// quotient by an IEEE division.  Otherwise x * inv, inv = 1 / scale rounded, which is off the
// quotient by less than 127 * 2^-22 < 2^-14: where it is nearer than that to halfway between two
// codes, the caller runs the exact form instead; d collects the largest distance from a code.
__device__ __forceinline__ void kv_codes8(const uint4& x, float inv, uint32_t (&c)[8], float& d) {
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, ties to even
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float f = __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
    const float t = fmaf(f, inv, kRound);
    c[i] = __float_as_uint(t);
    d = fmaxf(d, fabsf(fmaf(f, inv, kRound - t)));
  }
}

template <int kBits>
__device__ __forceinline__ void kv_codes8_exact(const uint4& x, float scale, uint32_t (&c)[8]) {
  constexpr float m = kBits == 8 ? 127.f : 7.f;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float f = __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
    // (a scale below the normal range can be far enough off max|x| / m to pass it)
    c[i] = static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(rintf(__fdiv_rn(f, scale)), -m), m)));
  }
}

template <int kBits>
__device__ __forceinline__ void kv_store8(uint8_t* dst, const uint32_t (&c)[8]) {
  if constexpr (kBits == 8) {
    uint2 o;
    o.x = prmt(prmt(c[0], c[1], 0x0040u), prmt(c[2], c[3], 0x0040u), 0x5410u);
    o.y = prmt(prmt(c[4], c[5], 0x0040u), prmt(c[6], c[7], 0x0040u), 0x5410u);
    *reinterpret_cast<uint2*>(dst) = o;
  } else {
    uint32_t o = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) o |= (c[i] & 15u) << (4 * i);
    *reinterpret_cast<uint32_t*>(dst) = o;
  }
}

template <int D, int kBits, bool kPaged>
__global__ void __launch_bounds__(256) fa_kv_write_kernel(const KvCopyParams p) {
  constexpr int kLanes = D / 16;         // lanes of one row
  constexpr int kRows = 32 / kLanes;     // rows the warp holds at once
  constexpr int kSteps = 32 / kRows;     // ... of the 32 it takes
  constexpr int kRow = D * kBits / 8;    // bytes of one row of codes
  constexpr float m = kBits == 8 ? 127.f : 7.f;
  const KvMap& map = p.map;
  if constexpr (kPaged) kv_check_cu(map);
  const int lane = threadIdx.x & 31;
  const long long unit = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int head = static_cast<int>(unit % map.Hkv);
  const long long rest = unit / map.Hkv;
  const bool is_v = rest & 1;
  const long long tok0 = (rest >> 1) * 32;
  if (tok0 >= map.N) return;
  const uint16_t* x = is_v ? p.v : p.k;
  const long long stride = is_v ? p.v_stride : p.k_stride;
  uint8_t* codes = is_v ? p.v_codes : p.k_codes;
  float* scales = is_v ? p.v_scale : p.k_scale;

  int page, row;  // of token tok0 + lane
  kv_locate<kPaged>(map, static_cast<int>(min(tok0 + lane, static_cast<long long>(map.N))), page,
                    row);
  float my_scale = 0.f;
  const int l = lane % kLanes;
#pragma unroll 1
  for (int s0 = 0; s0 < kSteps; s0 += 4) {
    uint4 w[4][2];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = (s0 + u) * kRows + lane / kLanes;
      w[u][0] = w[u][1] = make_uint4(0, 0, 0, 0);
      if (__shfl_sync(0xffffffffu, page, r) >= 0) {
        const uint4* src = reinterpret_cast<const uint4*>(x + (tok0 + r) * stride +
                                                          static_cast<long long>(head) * D);
        w[u][0] = __ldg(src + l);
        w[u][1] = __ldg(src + l + kLanes);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = (s0 + u) * kRows + lane / kLanes;
      const int pg = __shfl_sync(0xffffffffu, page, r);
      const int rw = __shfl_sync(0xffffffffu, row, r);
      // |bf16| as 16-bit integers keeps the order (infinity 0x7f80, NaN above)
      constexpr uint32_t kAbs = 0x7fff7fffu;
      uint32_t a = max_u16x2(max_u16x2(max_u16x2(w[u][0].x & kAbs, w[u][0].y & kAbs),
                                       max_u16x2(w[u][0].z & kAbs, w[u][0].w & kAbs)),
                             max_u16x2(max_u16x2(w[u][1].x & kAbs, w[u][1].y & kAbs),
                                       max_u16x2(w[u][1].z & kAbs, w[u][1].w & kAbs)));
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) a = max_u16x2(a, __shfl_xor_sync(0xffffffffu, a, o));
      a = max(a & 0xffffu, a >> 16);
      const bool finite = a < 0x7f80u;
      const float scale = finite ? __fdiv_rn(__uint_as_float(a << 16), m) : __int_as_float(0x7fc00000);
      // below this 1 / scale nears the end of the fp32 range: exact divisions
      const bool tiny = scale < 1e-30f;
      const bool zero = a == 0 || !finite;
      const float inv = (zero || tiny) ? 0.f : __frcp_rn(scale);
      uint32_t c0[8], c1[8];
      float d = 0.f;
      kv_codes8(w[u][0], zero ? 0.f : inv, c0, d);
      kv_codes8(w[u][1], zero ? 0.f : inv, c1, d);
      if (!zero && (tiny || d > 0.5f - 0x1p-14f)) {
        kv_codes8_exact<kBits>(w[u][0], scale, c0);
        kv_codes8_exact<kBits>(w[u][1], scale, c1);
      }
      if (!finite) {
#pragma unroll
        for (int i = 0; i < 8; ++i) c0[i] = c1[i] = 0;
      }
      const float s_lane = __shfl_sync(0xffffffffu, scale, (lane % kRows) * kLanes);
      if (lane / kRows == s0 + u) my_scale = s_lane;
      if (pg >= 0) {
        uint8_t* dst = codes + ((static_cast<size_t>(pg) * map.page_size + rw) * map.Hkv + head) * kRow;
        kv_store8<kBits>(dst + kBits * l, c0);
        kv_store8<kBits>(dst + kRow / 2 + kBits * l, c1);
      }
    }
  }
  if (page >= 0)
    scales[(static_cast<size_t>(page) * map.Hkv + head) * map.page_size + row] = my_scale;
}

// 8 codes -> bf16(code * scale).
template <int kBits>
__device__ __forceinline__ uint4 kv_values8(const uint8_t* src, float scale) {
  float f[8];
  if constexpr (kBits == 8) {
    const uint2 c = __ldg(reinterpret_cast<const uint2*>(src));
    // a byte x + 128 under the exponent of 2^23 is the float 2^23 + 128 + x
    const uint32_t w[2] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f[i] = __uint_as_float(prmt(w[i >> 2], 0x4B000000u, 0x7440u + (i & 3))) - 8388736.f;
  } else {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(src)) ^ 0x88888888u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f[i] = __uint_as_float(((w >> (4 * i)) & 15u) | 0x4B000000u) - 8388616.f;
  }
  uint4 o;
  o.x = pack_bf16x2(f[0] * scale, f[1] * scale);
  o.y = pack_bf16x2(f[2] * scale, f[3] * scale);
  o.z = pack_bf16x2(f[4] * scale, f[5] * scale);
  o.w = pack_bf16x2(f[6] * scale, f[7] * scale);
  return o;
}

template <int D, int kBits, bool kPaged>
__global__ void __launch_bounds__(256) fa_kv_read_kernel(const KvCopyParams p) {
  constexpr int kLanes = D / 16;
  constexpr int kRows = 32 / kLanes;
  constexpr int kSteps = 32 / kRows;
  constexpr int kRow = D * kBits / 8;
  const KvMap& map = p.map;
  if constexpr (kPaged) kv_check_cu(map);
  const int lane = threadIdx.x & 31;
  const long long unit = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int head = static_cast<int>(unit % map.Hkv);
  const long long rest = unit / map.Hkv;
  const bool is_v = rest & 1;
  const long long tok0 = (rest >> 1) * 32;
  if (tok0 >= map.N) return;
  const uint8_t* codes = is_v ? p.v_codes : p.k_codes;
  const float* scales = is_v ? p.v_scale : p.k_scale;
  uint16_t* out = is_v ? p.v_out : p.k_out;

  int page, row;
  kv_locate<kPaged>(map, static_cast<int>(min(tok0 + lane, static_cast<long long>(map.N))), page,
                    row);
  const float my_scale =
      page >= 0 ? scales[(static_cast<size_t>(page) * map.Hkv + head) * map.page_size + row] : 0.f;
  const int l = lane % kLanes;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int r = s * kRows + lane / kLanes;
    const int pg = __shfl_sync(0xffffffffu, page, r);
    const int rw = __shfl_sync(0xffffffffu, row, r);
    const float scale = __shfl_sync(0xffffffffu, my_scale, r);
    if (pg >= 0) {
      const uint8_t* src =
          codes + ((static_cast<size_t>(pg) * map.page_size + rw) * map.Hkv + head) * kRow;
      uint4* dst = reinterpret_cast<uint4*>(out + ((tok0 + r) * map.Hkv + head) * D);
      dst[l] = kv_values8<kBits>(src + kBits * l, scale);
      dst[l + kLanes] = kv_values8<kBits>(src + kRow / 2 + kBits * l, scale);
    }
  }
}

}  // namespace fa
