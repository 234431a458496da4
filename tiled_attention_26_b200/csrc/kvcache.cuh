// Writing the quantised KV cache and reading it back.
//
// A cache row is one token of one KV head.  The write maps its D bf16 values x to one fp32 scale
// and D codes ("Flash Attention on Ascend: three techniques", section 3, KV compression):
//   scale = fl32(max|x| / m)       code = clamp(rint(fl32(x / scale)), -m, m)       m = 127 or 7
// with ties to even and code 0 where the scale is 0; a row that holds an infinity or a NaN gets
// scale NaN and codes 0, so that whatever reads it is NaN rather than silently wrong.  The read
// is bf16(fl32(code * scale)).  Both move every byte once and are bound by HBM: 268 M elements written to
// INT8 in 130 us (6.3 TB/s, 0.96 of a copy's rate) and read back in 129; ragged tokens in pages reach 0.78
// of it (33 K tokens of 8 heads, 39 + 39 us), INT4 rows of 64 dims, 14 instructions an element, 0.6 (55 K tokens of
// 5 heads, 22.5 + 25; 21.4 + 25 where the rows are loaded before the offset that says how many there are is read).
//
// Both kernels see the cache as pages of P tokens: codes [page][P][Hkv][row bytes], scales
// [page][Hkv][P].  A contiguous cache [B, S, Hkv, ...] is the case P = S, page = sequence.
//
// Layout of the work: one warp takes 32 consecutive tokens of one KV head, of K or of V, so that
// the 32 scales (consecutive in memory) move as one coalesced access, lane = token (a small call: the
// tokens that the warp holds at once, so that more warps share it).  A row is
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

// Row of the code tensor, and element of the scale tensor, at `page`, `row` of a KV head.
__device__ __forceinline__ long long kv_row(const KvMap& m, int head, int page, int row) {
  return (static_cast<long long>(page) * m.page_size + row) * m.Hkv + head;
}
__device__ __forceinline__ long long kv_scale(const KvMap& m, int head, int page, int row) {
  return (static_cast<long long>(page) * m.Hkv + head) * m.page_size + row;
}

__device__ __forceinline__ long long shfl64(long long x, int from) {
  const uint32_t lo = __shfl_sync(0xffffffffu, static_cast<uint32_t>(x), from);
  const uint32_t hi = __shfl_sync(0xffffffffu, static_cast<uint32_t>(x >> 32), from);
  return static_cast<long long>(static_cast<unsigned long long>(hi) << 32 | lo);
}

// Of the `tokens` token rows from tok0 on, those that may be read: rows behind the last sequence need not exist.
__host__ __device__ inline int kv_rows_to_read(const KvMap& m, long long tok0, int tokens) {
  int end = m.N;
  if (m.cu_tokens != nullptr && m.cu_tokens[m.B] < end) end = m.cu_tokens[m.B];
  const long long left = end - tok0;
  return left <= 0 ? 0 : left < tokens ? static_cast<int>(left) : tokens;
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

// The codes of the 8 bf16 values in x as 8 bytes (INT8) or nibbles (INT4): rint(fl32(x / scale)),
// with inv = 1 / scale rounded and nscale = -scale.  The quotient comes from inv by one step of
// q + (x - q scale) inv (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  That leaves it off the rounded quotient by a unit in the last place at
// most; for scales that are a bf16 over m it rounds to the same code always (all pairs of mantissas and
// exponents, which is what the outcome depends on, are a test), x * inv alone does not: quotients on or
// next to a half are common, x = max / 2 is one.
// kTiny: x is multiplied by f first, as the scale was.  2^96 keeps the residuals of rows with scales
// below 2^-90 in the normal range (and changes no quotient); codes are clamped, for a scale below the
// normal range can be far enough off max|x| / m for the quotient to pass m.
template <int kBits, bool kTiny>
__device__ __forceinline__ uint2 kv_codes8(const uint4& x, float inv, float nscale, float f) {
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, ties to even
  constexpr float m = kBits == 8 ? 127.f : 7.f;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  const uint64_t inv2 = f2(inv, inv), ns2 = f2(nscale, nscale), round2 = f2(kRound, kRound);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint64_t v = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    if constexpr (kTiny) v = f2_mul(v, f2(f, f));
    uint64_t q = f2_mul(v, inv2);
    q = f2_fma(f2_fma(q, ns2, v), inv2, q);
    if constexpr (kTiny) {
      float a, b;
      f2_split(q, a, b);
      q = f2(fminf(fmaxf(a, -m), m), fminf(fmaxf(b, -m), m));
    }
    q = f2_add(q, round2);
    float a, b;
    f2_split(q, a, b);
    c[2 * i] = __float_as_uint(a);
    c[2 * i + 1] = __float_as_uint(b);
  }
  uint2 o;
  o.x = prmt(prmt(c[0], c[1], 0x0040u), prmt(c[2], c[3], 0x0040u), 0x5410u);
  o.y = prmt(prmt(c[4], c[5], 0x0040u), prmt(c[6], c[7], 0x0040u), 0x5410u);
  if constexpr (kBits == 4) {  // low nibbles of two bytes into one byte
    o.x &= 0x0f0f0f0fu;
    o.y &= 0x0f0f0f0fu;
    o.x = prmt(o.x | o.x >> 4, o.y | o.y >> 4, 0x6420u);
  }
  return o;
}

template <int kBits>
__device__ __forceinline__ void kv_store8(uint8_t* dst, const uint2& o) {
  if constexpr (kBits == 8)
    *reinterpret_cast<uint2*>(dst) = o;
  else
    *reinterpret_cast<uint32_t*>(dst) = o.x;
}

// kTokens: tokens of a warp, 32 (coalesced scales, one lookup of 32 places) or, for calls too small to
// fill the GPU that way, one step of 512 / D.
template <int D, int kBits, bool kPaged, int kTokens>
__global__ void __launch_bounds__(256) fa_kv_write_kernel(const KvCopyParams p) {
  constexpr int kLanes = D / 16;           // lanes of one row
  constexpr int kRows = 32 / kLanes;       // rows the warp holds at once
  constexpr int kSteps = kTokens / kRows;  // ... of the ones it takes
  constexpr int kU = kSteps < 4 ? kSteps : 4;  // steps in flight
  constexpr int kRow = D * kBits / 8;      // bytes of one row of codes
  constexpr float m = kBits == 8 ? 127.f : 7.f;
  const KvMap& map = p.map;
  const int lane = threadIdx.x & 31;
  const uint32_t unit = blockIdx.x * 8 + (threadIdx.x >> 5);  // (fewer than 2^32: the launch checks)
  const int head = static_cast<int>(unit % static_cast<uint32_t>(map.Hkv));
  const uint32_t rest = unit / static_cast<uint32_t>(map.Hkv);
  const bool is_v = rest & 1;
  const long long tok0 = static_cast<long long>(rest >> 1) * kTokens;
  if constexpr (kPaged) kv_check_cu(map);
  const int left = kv_rows_to_read(map, tok0, kTokens);
  if (left == 0) return;
  const long long stride = is_v ? p.v_stride : p.k_stride;
  const uint16_t* x = (is_v ? p.v : p.k) + tok0 * stride + static_cast<long long>(head) * D;
  uint8_t* codes = is_v ? p.v_codes : p.k_codes;
  float* scales = is_v ? p.v_scale : p.k_scale;

  const int l = lane % kLanes;
  uint4 w[kU][2];
  auto load = [&](int s0) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int r = (s0 + u) * kRows + lane / kLanes;
      w[u][0] = w[u][1] = make_uint4(0, 0, 0, 0);
      if (r < left) {
        const uint4* src = reinterpret_cast<const uint4*>(x + r * stride);
        w[u][0] = __ldg(src + l);
        w[u][1] = __ldg(src + l + kLanes);
      }
    }
  };
  load(0);  // (on its way while the places are looked up)
  int page = -1, row = 0;  // of token tok0 + lane
  if (lane < left) kv_locate<kPaged>(map, static_cast<int>(tok0) + lane, page, row);
  const long long at = page < 0 ? -1 : kv_row(map, head, page, row);
  float my_scale = 0.f;
#pragma unroll 1
  for (int s0 = 0; s0 < kSteps; s0 += kU) {
    if (s0 > 0) load(s0);
    // lane l < kU of a row's lanes takes the scale of step s0 + l
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      // |bf16| as 16-bit integers keeps the order (infinity 0x7f80, NaN above)
      constexpr uint32_t kAbs = 0x7fff7fffu;
      uint32_t a = __vmaxu2(__vmaxu2(__vmaxu2(w[u][0].x & kAbs, w[u][0].y & kAbs),
                                     __vmaxu2(w[u][0].z & kAbs, w[u][0].w & kAbs)),
                            __vmaxu2(__vmaxu2(w[u][1].x & kAbs, w[u][1].y & kAbs),
                                     __vmaxu2(w[u][1].z & kAbs, w[u][1].w & kAbs)));
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) a = __vmaxu2(a, __shfl_xor_sync(0xffffffffu, a, o));
      if (l % kU == u) top = max(a & 0xffffu, a >> 16);
    }
    const bool finite = top < 0x7f80u;
    const float scale = finite ? __fdiv_rn(__uint_as_float(top << 16), m) : __int_as_float(0x7fc00000);
    const bool tiny = scale < 0x1p-90f && top != 0;
    const bool any_tiny = __any_sync(0xffffffffu, tiny);
    const float f = tiny ? 0x1p96f : 1.f;
    const float base = scale * f;
    // 1 / scale = 0 makes every code 0
    const float inv = (top == 0 || !finite) ? 0.f : __frcp_rn(base);
    const float from = __shfl_sync(0xffffffffu, scale, lane % kRows * kLanes + lane / kRows % kU);
    if (lane / kRows / kU == s0 / kU) my_scale = from;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int r = (s0 + u) * kRows + lane / kLanes;
      const long long to = shfl64(at, r & 31);
      const float inv_u = __shfl_sync(0xffffffffu, inv, lane / kLanes * kLanes + u);
      const float ns_u = -__shfl_sync(0xffffffffu, base, lane / kLanes * kLanes + u);
      uint2 c0, c1;
      if (!any_tiny) {
        c0 = kv_codes8<kBits, false>(w[u][0], inv_u, ns_u, 1.f);
        c1 = kv_codes8<kBits, false>(w[u][1], inv_u, ns_u, 1.f);
      } else {
        const float f_u = __shfl_sync(0xffffffffu, f, lane / kLanes * kLanes + u);
        c0 = kv_codes8<kBits, true>(w[u][0], inv_u, ns_u, f_u);
        c1 = kv_codes8<kBits, true>(w[u][1], inv_u, ns_u, f_u);
      }
      if (inv_u == 0.f) c0 = c1 = make_uint2(0, 0);
      if (to >= 0) {
        uint8_t* dst = codes + to * kRow;
        kv_store8<kBits>(dst + kBits * l, c0);
        kv_store8<kBits>(dst + kRow / 2 + kBits * l, c1);
      }
    }
  }
  if (page >= 0)
    scales[kv_scale(map, head, page, row)] = my_scale;
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

template <int D, int kBits, bool kPaged, int kTokens>
__global__ void __launch_bounds__(256) fa_kv_read_kernel(const KvCopyParams p) {
  constexpr int kLanes = D / 16;
  constexpr int kRows = 32 / kLanes;
  constexpr int kSteps = kTokens / kRows;
  constexpr int kRow = D * kBits / 8;
  const KvMap& map = p.map;
  if constexpr (kPaged) kv_check_cu(map);
  const int lane = threadIdx.x & 31;
  const uint32_t unit = blockIdx.x * 8 + (threadIdx.x >> 5);  // (fewer than 2^32: the launch checks)
  const int head = static_cast<int>(unit % static_cast<uint32_t>(map.Hkv));
  const uint32_t rest = unit / static_cast<uint32_t>(map.Hkv);
  const bool is_v = rest & 1;
  const long long tok0 = static_cast<long long>(rest >> 1) * kTokens;
  if (tok0 >= map.N) return;
  const int left = static_cast<int>(min(static_cast<long long>(kTokens), map.N - tok0));
  const uint8_t* codes = is_v ? p.v_codes : p.k_codes;
  const float* scales = is_v ? p.v_scale : p.k_scale;
  uint16_t* out = is_v ? p.v_out : p.k_out;

  int page = -1, row = 0;
  if (lane < left) kv_locate<kPaged>(map, static_cast<int>(tok0) + lane, page, row);
  const float my_scale =
      page >= 0 ? scales[kv_scale(map, head, page, row)] : 0.f;
  const long long at = page < 0 ? -1 : kv_row(map, head, page, row);
  const int l = lane % kLanes;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int r = s * kRows + lane / kLanes;
    const long long from = shfl64(at, r);
    const float scale = __shfl_sync(0xffffffffu, my_scale, r);
    if (from >= 0) {
      const uint8_t* src = codes + from * kRow;
      uint4* dst = reinterpret_cast<uint4*>(out + ((tok0 + r) * map.Hkv + head) * D);
      dst[l] = kv_values8<kBits>(src + kBits * l, scale);
      dst[l + kLanes] = kv_values8<kBits>(src + kRow / 2 + kBits * l, scale);
    }
  }
}

}  // namespace fa
