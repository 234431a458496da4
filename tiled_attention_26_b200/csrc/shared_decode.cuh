// Decode attention over a prefix that every sequence of the batch shares.
//
// One query token per sequence, B sequences, G query heads per KV head: the R = B * G query rows
// of a KV head all attend to the same prefix keys, so the prefix part of the attention is a
// matrix product with R rows per staged K/V tile instead of G, and the cache is read once instead
// of B times:
//   x_rj = scale * k_scale_j * (q_r . kcode_j),   O_r = sum_j p_rj * v_scale_j * vcode_j
// (the codes take part without being decompressed first: "Flash Attention on Ascend: three
// techniques", section 3).  The keys each sequence owns go through the paged split kernel of
// decode.cuh; both write partial outputs with their log-sum-exp, and fa_decode_combine_kernel
// merges them: L = log sum_s exp(L_s), O = sum_s exp(L_s - L) O_s.
//
// fa_shared_prefix_kernel, one CTA per (KV head, block of 128 rows, split of the prefix), 512 threads:
//   warps 0-7   two softmax warpgroups that take the key tiles in turn (thread = query row = TMEM lane)
//   warps 8-11  dequantisation: thread = key; K codes to fp16 (exact), V codes times their scale to
//               fp16, both into the swizzled layout the tensor core reads
//   warp 12     TMA producer: K and V code tiles of 128 keys, one box per page piece
//   warp 13     allocates TMEM and issues tcgen05.mma from one thread: S_j = Q K_j^T, O += P_j V_j
//               with P_j from TMEM, over S_j's columns
//   warp 14     the keys' scales, and the exponent E below;  warp 15 idles
// S has three buffers in TMEM and O one (3 * 128 + D columns): while the warpgroups work on tiles j and
// j + 1, the tensor core computes S_{j+2}, so no softmax waits for a product of its own.  One
// accumulator means one running maximum per row: it goes from warpgroup to warpgroup with the tiles,
// through shared memory, before the exponentials.  (Two accumulators of 128 rows, or one each for two
// streams of tiles, leave room for two S buffers only, and every softmax then waited for its
// own P V and the next Q K^T: 5.1 thousand cycles for 2 x 128 x 128 scores at D = 128.)
//
// Number formats.  Q is scaled per row by a power of two and kept in fp16, which holds a bf16 row
// exactly (elements more than 2^29 below the row's largest lose bits).  Scores, maxima, sums, O and
// log-sum-exps are fp32; k_scale multiplies the fp32 scores, so QK^T has no rounding of its
// own.  P = 2^7 p (p <= 2^8 with the lazy maximum) and v_scale * vcode * 2^E are rounded to fp16
// (relative 2^-11 each, an eighth of the bf16 output's): the shift by 2^7 keeps weights down to
// 2^-31 of the maximum from vanishing, and the power E, lowered (with an exact rescale of O) when a
// larger v_scale arrives, keeps V below 2^15.
#pragma once

#include "decode.cuh"
#include "sm100.cuh"

namespace fa {

struct SharedParams {
  const uint16_t* q;  // bf16 [B, 1, Hq, D]
  const float* k_scale;  // [num_pages, Hkv, P]
  const float* v_scale;
  const int32_t* table;  // [max_pages] pages of the prefix
  const int32_t* len;    // [1] keys of the prefix
  float* o_part;         // [splits, B, Hq, D]
  float* lse_part;       // [splits, B, Hq] natural log
  int B, Hq, Hkv, G, R, row_blocks, splits;
  int max_pages, num_pages, page_shift;
  float scale_log2;
  uint64_t timeout_ns;
};

template <int D, int kBits>
struct SharedCfg {
  static constexpr int kThreads = 512;
  static constexpr int kRow = D * kBits / 8;       // bytes of one row of codes
  static constexpr int kAtom = 128 * 128;          // 128 rows x 128 bytes (64 fp16)
  static constexpr int kTile = 128 * D * 2;        // 128 rows of fp16
  static constexpr int kRawTile = 128 * kRow;
  static constexpr int kRaw = 2;                   // stages of code tiles
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kTile;              // [2]
  static constexpr int kVOff = kKOff + 2 * kTile;  // [2]
  static constexpr int kRawKOff = kVOff + 2 * kTile;
  static constexpr int kRawVOff = kRawKOff + kRaw * kRawTile;
  static constexpr int kKsOff = kRawVOff + kRaw * kRawTile;  // fp32 k_scale [3 tiles][128]
  static constexpr int kVsOff = kKsOff + 3 * 512;            // fp16 v_scale * 2^E [2 tiles][128]
  static constexpr int kMaxOff = kVsOff + 2 * 256;           // fp32 [128] rows' running maximum
  static constexpr int kExpOff = kMaxOff + 512;              // int [3 tiles][E, E of the tile before]
  static constexpr int kBarOff = kExpOff + 32;
  static constexpr int kBarQ = 0;
  static constexpr int kBarRawKFull = 1;             // [kRaw]
  static constexpr int kBarRawVFull = kBarRawKFull + kRaw;
  static constexpr int kBarRawKEmpty = kBarRawVFull + kRaw;
  static constexpr int kBarRawVEmpty = kBarRawKEmpty + kRaw;
  static constexpr int kBarKFull = kBarRawVEmpty + kRaw;  // [2]
  static constexpr int kBarVFull = kBarKFull + 2;
  static constexpr int kBarKEmpty = kBarVFull + 2;
  static constexpr int kBarVEmpty = kBarKEmpty + 2;
  static constexpr int kBarKs = kBarVEmpty + 2;      // [3] k_scale and E
  static constexpr int kBarVs = kBarKs + 3;          // [2]
  static constexpr int kBarSFull = kBarVs + 2;       // [3]
  static constexpr int kBarPFull = kBarSFull + 3;    // [3][2 halves]
  static constexpr int kBarMax = kBarPFull + 6;      // [2 warpgroups][4 warps]
  static constexpr int kBarOFinal = kBarMax + 8;
  static constexpr int kBarDrain = kBarOFinal + 1;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr int kMiscOff = kBarOff + 8 * kNumBars;
  static constexpr int kSmemBytes = kMiscOff + 16;
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColO = 3 * 128;  // S buffer b at column 128 b
};

// Instruction descriptor for kind::f16 with fp16 A/B and an fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t(N) >> 3) << 17) |
         ((uint32_t(M) >> 4) << 24);
}

// Largest exponent e with x * 2^e < 2^top (x >= 0), kept where 2^e and 2^-e are normal fp32 numbers.
__device__ __forceinline__ int exponent_below(float x, int top) {
  const int ex = static_cast<int>((__float_as_uint(x) >> 23) & 255u) - 126;  // x < 2^ex
  return max(-120, min(120, top - ex));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

// The 16-bit value at addr, twice.
__device__ __forceinline__ uint32_t lds16x2(uint32_t addr) {
  uint16_t x;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(addr));
  return prmt(x, x, 0x1010u);
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t a) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(a) : "memory");
}

// One key's row of codes (in the raw tile, swizzled by its TMA box) times vs (an fp16 pair) to fp16 in
// the layout of a tensor-core operand: 64-dim atoms of 128-byte rows, 16-byte chunk index XOR row % 8.
// INT4: within each 8-dim chunk the dims stand in the order 0, 4, 2, 6, 1, 5, 3, 7 (that of the
// nibble extraction); the last four come out as 16 x the code, which vs_hi = vs / 16 or the other
// operand undoes.
template <int D, int kBits>
__device__ __forceinline__ void dequant_row(uint32_t raw, uint32_t dst, int r, uint32_t vs,
                                            uint32_t vs_hi) {
  constexpr int kRow = D * kBits / 8;
  const uint32_t row = dst + r * 128;
  auto put = [&](int chunk, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    sts128(row + (chunk >> 3) * (128 * 128) + (((chunk & 7) ^ (r & 7)) << 4), mul_f16x2(a, vs),
           mul_f16x2(b, vs), mul_f16x2(c, vs_hi), mul_f16x2(d, vs_hi));
  };
  constexpr int kLoads = kRow / 16 < 4 ? kRow / 16 : 4;  // in flight
#pragma unroll 1
  for (int c0 = 0; c0 < kRow / 16; c0 += kLoads) {
    uint4 x[kLoads];
#pragma unroll
    for (int c = 0; c < kLoads; ++c) x[c] = lds128(raw + swz<kRow>(r * kRow + 16 * (c0 + c)));
#pragma unroll
    for (int c = 0; c < kLoads; ++c) {
      const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
      if constexpr (kBits == 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t u = w[2 * h] ^ 0x80808080u, v = w[2 * h + 1] ^ 0x80808080u;
          put(2 * (c0 + c) + h, codes_to_f16x2(u, kSelB01), codes_to_f16x2(u, kSelB23),
              codes_to_f16x2(v, kSelB01), codes_to_f16x2(v, kSelB23));
        }
      } else {
#pragma unroll
        for (int h = 0; h < 4; ++h)
          put(4 * (c0 + c) + h, nib_lo_f16x2(w[h]), nib_lo_f16x2(w[h] >> 8), nib_hi16_f16x2(w[h]),
              nib_hi16_f16x2(w[h] >> 8));
      }
    }
  }
}

template <int D, int kBits>
__global__ void __launch_bounds__(512, 1)
    fa_shared_prefix_kernel(const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const SharedParams p) {
  using C = SharedCfg<D, kBits>;
  asm volatile("griddepcontrol.launch_dependents;");  // (the merge waits on the device)
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // the swizzled tiles need 1024-byte aligned shared memory, and there is no room to align it here
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(&g_fa_device_status, kDevStatusLayout);
    return;
  }
  uint8_t* smem = smem_raw;
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int idx) { return sb + C::kBarOff + 8u * idx; };
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  int* abort_flag = reinterpret_cast<int*>(smem + C::kMiscOff + 4);
  const WaitCtl ctl{abort_flag, p.timeout_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // KV heads vary fastest, then row blocks: CTAs that run together read the same key rows
  const int kvh = static_cast<int>(blockIdx.x) % p.Hkv;
  const int rb = static_cast<int>(blockIdx.x) / p.Hkv % p.row_blocks;
  const int split = static_cast<int>(blockIdx.x) / (p.Hkv * p.row_blocks);
  const int row0 = rb * 128;
  const int live = min(128, p.R - row0);  // query rows of this CTA

  int len = p.len[0];
  {
    const int cap = p.max_pages << p.page_shift;
    if (len < 0 || len > cap) {
      if (threadIdx.x == 0) atomicOr(&g_fa_device_status, kDevStatusBadIndex);
      len = max(0, min(len, cap));
    }
  }
  // splits are whole tiles, as even as they come: the first `extra` splits take one more
  const int tiles = (len + 127) / 128;
  const int per = tiles / p.splits, extra = tiles % p.splits;
  const int t_begin = (split * per + min(split, extra)) * 128;
  const int nt = per + (split < extra ? 1 : 0);
  const int t_end = min(len, t_begin + 128 * nt);

  // query row r of this CTA: head kvh * G + (row0 + r) % G of sequence (row0 + r) / G
  auto out_row = [&](int r) -> size_t {
    const int x = row0 + r;
    return static_cast<size_t>(x / p.G) * p.Hq + static_cast<size_t>(kvh) * p.G + x % p.G;
  };
  const size_t rows = static_cast<size_t>(p.B) * p.Hq;
  if (nt == 0) {
    for (int r = threadIdx.x; r < live; r += blockDim.x)
      p.lse_part[split * rows + out_row(r)] = -INFINITY;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // (as below)
    return;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kNumBars; ++i) {
      uint32_t count = 1;
      if (i == C::kBarQ) count = 256;
      if (i >= C::kBarPFull && i < C::kBarMax) count = (live + 31) / 32 * 32;  // warps with a row
      if (i >= C::kBarRawKEmpty && i < C::kBarKEmpty) count = 4;
      mbar_init(bar(i), count);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 12 && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 13) {
    tmem_alloc(smem_u32(tmem_holder), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  auto checked_page = [&](int pg) -> int {
    if (static_cast<unsigned>(pg) >= static_cast<unsigned>(p.num_pages)) {
      atomicOr(&g_fa_device_status, kDevStatusBadIndex);
      pg = 0;
    }
    return pg;
  };

  if (warp >= 12) {
    if (warp == 12) {
      // ================= TMA producer =================
      // lane i < boxes copies box i of each tile (a page, or 128 keys of a larger one); boxes past
      // the last key are skipped: the codes left there are finite and their scales count as 0
      const int box_t = min(128, 1 << p.page_shift);
      const int boxes = 128 / box_t;
      const int pmask = (1 << p.page_shift) - 1;
      const uint32_t box_bytes = static_cast<uint32_t>(box_t) * C::kRow;
      const uint64_t pol = l2_evict_first_policy();
      auto entry_at = [&](int j) -> int {
        const int t = t_begin + 128 * j + lane * box_t;
        return lane < boxes && j < nt && t < t_end ? __ldg(p.table + (t >> p.page_shift)) : 0;
      };
      int entry = entry_at(0), issued = 0;
      bool ok = true;
      for (int j = 0; j < nt && ok; ++j) {
        const int next = entry_at(j + 1);
        const int s = j % C::kRaw, ph = (j / C::kRaw) & 1;
        const int t = t_begin + 128 * j + lane * box_t;
        const int pg = lane < boxes && t < t_end ? checked_page(entry) : -1;
        const uint32_t n_live = __popc(__ballot_sync(0xffffffffu, pg >= 0));
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
          const uint32_t full = bar((kind ? C::kBarRawVFull : C::kBarRawKFull) + s);
          ok = ok && mbar_wait(bar((kind ? C::kBarRawVEmpty : C::kBarRawKEmpty) + s), ph ^ 1, ctl);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(full, n_live * box_bytes);
          __syncwarp();
          const uint32_t dst = sb + (kind ? C::kRawVOff : C::kRawKOff) + s * C::kRawTile +
                               lane * box_t * C::kRow;
          if (pg >= 0) {
            // several row blocks read the prefix: let it stay in L2 for them
            if (p.row_blocks > 1)
              tma_load_4d(dst, kind ? &tm_v : &tm_k, full, 0, kvh, t & pmask, pg);
            else
              tma_load_4d_policy(dst, kind ? &tm_v : &tm_k, full, 0, kvh, t & pmask, pg, pol);
          }
          issued = 2 * j + kind + 1;
        }
        entry = next;
      }
      // Every copy this warp started has landed before the CTA can exit (already true unless a
      // consumer gave up; then this waits, bounded).
      __syncwarp();
      if (lane == 0) {
        volatile int zero = 0;
        const WaitCtl drain_ctl{&zero, p.timeout_ns};
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
          const int n = (issued + 1 - kind) / 2;  // tiles of this kind
          for (int s = 0; s < C::kRaw && s < n; ++s)
            mbar_wait(bar((kind ? C::kBarRawVFull : C::kBarRawKFull) + s),
                      ((n - 1 - s) / C::kRaw) & 1, drain_ctl);
        }
      }
    } else if (warp == 14) {
      // ================= scales: lane i has keys 4 i .. 4 i + 3 of each tile =================
      // k_scale as it is, v_scale times 2^E; keys past the prefix count 0.  Table entries are read two
      // tiles ahead, scales one ahead.
      const int pmask = (1 << p.page_shift) - 1;
      auto entry_at = [&](int j) -> int {
        const int t = t_begin + 128 * j + 4 * lane;
        return j < nt && t < t_end ? __ldg(p.table + (t >> p.page_shift)) : 0;
      };
      auto scales_at = [&](int j, int entry, float4& ks, float4& vs) {
        const int t = t_begin + 128 * j + 4 * lane;
        ks = vs = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j < nt && t < t_end) {
          const size_t at =
              ((static_cast<size_t>(checked_page(entry)) * p.Hkv + kvh) << p.page_shift) + (t & pmask);
          ks = __ldg(reinterpret_cast<const float4*>(p.k_scale + at));
          vs = __ldg(reinterpret_cast<const float4*>(p.v_scale + at));
        }
      };
      float4 ks, vs, ks_next, vs_next;
      scales_at(0, entry_at(0), ks, vs);
      int entry = entry_at(1);
      constexpr int kUnset = 1 << 20;
      int e_old = kUnset;
      for (int j = 0; j < nt; ++j) {
        scales_at(j + 1, entry, ks_next, vs_next);
        entry = entry_at(j + 2);
        const int left = t_end - (t_begin + 128 * j + 4 * lane);
        if (left < 4) {  // the page's scales behind the prefix may be anything
          if (left < 1) ks.x = vs.x = 0.f;
          if (left < 2) ks.y = vs.y = 0.f;
          if (left < 3) ks.z = vs.z = 0.f;
          ks.w = vs.w = 0.f;
        }
        const uint32_t kAbs = 0x7fffffffu;
        const uint32_t top = __reduce_max_sync(
            0xffffffffu, max(max(__float_as_uint(vs.x) & kAbs, __float_as_uint(vs.y) & kAbs),
                             max(__float_as_uint(vs.z) & kAbs, __float_as_uint(vs.w) & kAbs)));
        const int e = min(e_old, exponent_below(__uint_as_float(top), 8));
        const float f = exp2i(e);
        // k_scale's slot is free once the probabilities of tile j - 3 are there, v_scale's once the
        // products of tile j - 2 are done
        bool ok = mbar_wait(bar(C::kBarPFull + 2 * (j % 3) + 1), ((j / 3) & 1) ^ 1, ctl);
        if (!__all_sync(0xffffffffu, ok)) break;
        sts128(sb + C::kKsOff + j % 3 * 512 + 16 * lane, __float_as_uint(ks.x), __float_as_uint(ks.y),
               __float_as_uint(ks.z), __float_as_uint(ks.w));
        if (lane == 0) sts64(sb + C::kExpOff + 8 * (j % 3), e, j == 0 ? e : e_old);
        e_old = e;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kBarKs + j % 3));
        ok = mbar_wait(bar(C::kBarVEmpty + (j & 1)), ((j >> 1) & 1) ^ 1, ctl);
        if (!__all_sync(0xffffffffu, ok)) break;
        sts64(sb + C::kVsOff + (j & 1) * 256 + 8 * lane, pack_f16x2(vs.x * f, vs.y * f),
              pack_f16x2(vs.z * f, vs.w * f));
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kBarVs + (j & 1)));
        ks = ks_next;
        vs = vs_next;
      }
    } else if (warp == 13) {
      // ================= MMA issuer =================
      constexpr uint32_t idesc_qk = idesc_f16_f32(128, 128, false);
      constexpr uint32_t idesc_pv = idesc_f16_f32(128, D, true);
      // The whole warp runs the loop and one lane's instructions count: in code that one lane alone runs
      // the operands of each product went through vector registers.
      const bool one = elect_one();
      // operand descriptors differ in the address field only (16-byte units, low word): one add each
      const uint64_t desc_k_major = smem_desc_sw128(0, 16, 1024);
      const uint64_t desc_v = smem_desc_sw128(0, C::kAtom, 1024);
      auto wait = [&](int b, int parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, ctl));
      };
      auto issue_qk = [&](int buf, int slot) {
        const uint32_t qa = (sb + C::kQOff) >> 4;
        const uint32_t kb = (sb + C::kKOff + slot * C::kTile) >> 4;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk / 4) * C::kAtom + (kk % 4) * 32) >> 4;
          umma_ss_if(tmem + 128 * buf, desc_k_major + (qa + off), desc_k_major + (kb + off), idesc_qk,
                  kk > 0 ? 1u : 0u, one);
        }
        tc_commit_if(bar(C::kBarSFull + buf), one);
        tc_commit_if(bar(C::kBarKEmpty + slot), one);
      };
      // O += P_j V_j; P_j arrives in two halves of 64 keys
      auto issue_pv = [&](int j, int buf, int use) -> bool {
        const uint32_t vb = (sb + C::kVOff + (j & 1) * C::kTile) >> 4;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!wait(C::kBarPFull + 2 * buf + half, use & 1)) return false;
          tc_fence_after();
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {
            const int kk = 4 * half + k4;
            umma_ts_if(tmem + C::kColO, tmem + 128 * buf + kk * 8, desc_v + (vb + kk * 128), idesc_pv,
                    (j == 0 && kk == 0) ? 0u : 1u, one);
          }
        }
        return true;
      };
      // tile j sits in slot j & 1 of K and V, in that slot's use number j >> 1, and in buffer j % 3 of S
      bool ok = wait(C::kBarQ, 0);
      int buf = 0;  // of the next tile of S
#pragma unroll 1  // (one copy of the issue code: more do not fit this warp's registers)
      for (int j = -2; j < nt && ok; ++j) {
        // S_{j+2} over P_{j-1}, whose products are already issued
        if (j + 2 < nt) {
          ok = wait(C::kBarKFull + (j & 1), ((j + 2) >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          issue_qk(buf, j & 1);
        }
        buf = buf == 2 ? 0 : buf + 1;
        if (j < 0) continue;
        ok = wait(C::kBarVFull + (j & 1), (j >> 1) & 1) && issue_pv(j, buf, j / 3);
        if (!ok) break;
        tc_commit_if(bar(C::kBarVEmpty + (j & 1)), one);
        if (j + 1 == nt) tc_commit_if(bar(C::kBarOFinal), one);
      }
      // Drain: every MMA this thread issued has completed before TMEM is released.
      tc_commit_if(bar(C::kBarDrain), one);
      volatile int zero = 0;
      const WaitCtl drain_ctl{&zero, p.timeout_ns};
      mbar_wait(bar(C::kBarDrain), 0, drain_ctl);
    }
  } else if (warp >= 8) {
    // ================= dequantisation: thread r = key r of each tile =================
    const int r = threadIdx.x & 127;
    // K_0, K_1, V_0, K_2, V_1, ...: V_j's slot is free only after the products of tile j - 2, and K_{j+1}
    // must not wait for that.  (K's codes times 1: one copy of the code for both, see below.)
#pragma unroll 1
    for (int i = 0; i < 2 * nt + 2; ++i) {
      const int kind = i & 1, j = (i >> 1) - kind;
      if (j < 0 || j >= nt) continue;
      const int slot = j & 1, use = (j >> 1) & 1;
      // (V's scales are written after V's slot is free)
      const bool ok = mbar_wait(bar((kind ? C::kBarVs : C::kBarKEmpty) + slot), use ^ kind ^ 1, ctl) &&
                      mbar_wait(bar((kind ? C::kBarRawVFull : C::kBarRawKFull) + slot), use, ctl);
      if (!__all_sync(0xffffffffu, ok)) break;
      const uint32_t vs = kind ? lds16x2(sb + C::kVsOff + slot * 256 + 2 * r) : 0x3C003C00u;
      dequant_row<D, kBits>(sb + (kind ? C::kRawVOff : C::kRawKOff) + slot * C::kRawTile,
                            sb + (kind ? C::kVOff : C::kKOff) + slot * C::kTile, r, vs,
                            kBits == 4 && kind ? mul_f16x2(vs, 0x2C002C00u) : vs);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar((kind ? C::kBarRawVEmpty : C::kBarRawKEmpty) + slot));
        mbar_arrive(bar((kind ? C::kBarVFull : C::kBarKFull) + slot));
      }
    }
  } else {
    // ================= Q, softmax, epilogue: thread = query row r, warpgroup t =================
    const int t = warp >> 2, w4 = warp & 3;
    const int r = threadIdx.x & 127;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * w4) << 16);
    const bool warp_live = 32 * w4 < live;  // a warp of padding rows only writes out

    // Both warpgroups read the same rows (warp w of each rows 32 (w % 4) .. + 31, D / 8 lanes a row) and
    // lay out half of them.
    constexpr int kQLanes = D / 8, kQRows = 32 / kQLanes, kQSteps = 32 / kQRows;
    const int my_row = static_cast<int>(out_row(min(32 * w4 + lane, live - 1)));
    float sc = 0.f;  // of row r: score units of log2, undoing the row's power of two
#pragma unroll 1
    for (int i0 = 0; i0 < kQSteps; i0 += 8) {
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = (i0 + i) * kQRows + lane / kQLanes;
      const size_t from = __shfl_sync(0xffffffffu, my_row, row);
      x[i] = make_uint4(0, 0, 0, 0);
      if (32 * w4 + row < live)
        x[i] = __ldg(reinterpret_cast<const uint4*>(p.q + from * D) + lane % kQLanes);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = 32 * w4 + (i0 + i) * kQRows + lane / kQLanes, c = lane % kQLanes;
      const uint32_t kAbs = 0x7fff7fffu;
      uint32_t am = __vmaxu2(__vmaxu2(x[i].x & kAbs, x[i].y & kAbs), __vmaxu2(x[i].z & kAbs, x[i].w & kAbs));
#pragma unroll
      for (int o = 1; o < kQLanes; o <<= 1) am = __vmaxu2(am, __shfl_xor_sync(0xffffffffu, am, o));
      const int eq = exponent_below(__uint_as_float(max(am & 0xffffu, am >> 16) << 16), 15);
      // (not 0: a masked score is -infinity times this)
      const float sc_i = __shfl_sync(0xffffffffu, fmaxf(p.scale_log2 * exp2i(-eq), 0x1p-126f),
                                     lane % kQRows * kQLanes);
      if (lane / kQRows == i0 + i) sc = sc_i;
      if ((i & 1) != t) continue;  // each warpgroup lays out half of the rows
      const float qs = exp2i(eq);
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      float f[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[2 * k] = __uint_as_float(w[k] << 16) * qs;
        f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u) * qs;
      }
      uint32_t h[4];
      if constexpr (kBits == 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = pack_f16x2(f[2 * k], f[2 * k + 1]);
      } else {  // the K operand's dim order, and 1/16 for its 16 x codes
        h[0] = pack_f16x2(f[0], f[4]);
        h[1] = pack_f16x2(f[2], f[6]);
        h[2] = pack_f16x2(f[1] * 0.0625f, f[5] * 0.0625f);
        h[3] = pack_f16x2(f[3] * 0.0625f, f[7] * 0.0625f);
      }
      sts128(sb + C::kQOff + (c >> 3) * C::kAtom + row * 128 + (((c & 7) ^ (row & 7)) << 4), h[0], h[1],
             h[2], h[3]);
    }
    }
    fence_proxy_async_smem();
    mbar_arrive(bar(C::kBarQ));

    // The running maximum after tile j - 1 (of the other warpgroup) and its barrier.
    const uint32_t m_at = sb + C::kMaxOff + 4 * r;
    auto max_wait = [&](int j) {  // of tile j
      return mbar_wait(bar(C::kBarMax + 4 * (j & 1) + w4), (j >> 1) & 1, ctl);
    };
    float m = -INFINITY, l = 0.f;  // l: of this warpgroup's tiles, relative to m
    int buf = t;
    bool ok = true;
    for (int j = t; warp_live && j < nt; j += 2) {  // (a warp of padding rows has nothing to do)
      const int b = buf, use = (j / 3) & 1;  // buffer of S, k_scale and P
      ok = mbar_wait(bar(C::kBarSFull + b), use, ctl);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t colS = trow + 128 * b;
      buf = buf == 0 ? 2 : buf - 1;  // (j + 2) % 3
      ok = mbar_wait(bar(C::kBarKs + b), use, ctl);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      // S is read twice, for the maximum and for the probabilities, 32 columns at a time in rolled loops,
      // a load ahead of the arithmetic.  (Kept in registers between the two it takes unrolled code, and
      // with the other warps' loops that no longer fitted the instruction caches: half of all
      // stalls waited for instructions.)
      uint32_t s0[32], s1[32];
      tmem_ld32(colS, s0);
      const uint2 ee = lds64(sb + C::kExpOff + 8 * b);
      const int e_new = static_cast<int>(ee.x), e_old = static_cast<int>(ee.y);
      const int limit = t_end - (t_begin + 128 * j);
      const uint32_t ring = sb + C::kKsOff + b * 512;
      // scores of 32 keys: S times k_scale (the row's common factor sc joins in the exponent)
      auto scores = [&](uint32_t (&v)[32], int c) {
#pragma unroll
        for (int q4 = 0; q4 < 8; ++q4) {
          const uint4 k4 = lds128(ring + 128 * c + 16 * q4);
          uint32_t* y = v + 4 * q4;
          float a0, a1, b0, b1;
          f2_split(f2_mul(f2(__uint_as_float(y[0]), __uint_as_float(y[1])),
                          f2(__uint_as_float(k4.x), __uint_as_float(k4.y))), a0, a1);
          f2_split(f2_mul(f2(__uint_as_float(y[2]), __uint_as_float(y[3])),
                          f2(__uint_as_float(k4.z), __uint_as_float(k4.w))), b0, b1);
          y[0] = __float_as_uint(a0);
          y[1] = __float_as_uint(a1);
          y[2] = __float_as_uint(b0);
          y[3] = __float_as_uint(b1);
        }
        if (limit < 32 * c + 32) {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (32 * c + k >= limit) v[k] = __float_as_uint(-INFINITY);
        }
      };
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      auto maximum = [&](uint32_t (&v)[32], int c) {
        scores(v, c);
#pragma unroll
        for (int k = 0; k < 16; ++k)
          mx[k & 3] = fmax3(mx[k & 3], __uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]));
      };
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        tmem_wait_ld();
        tmem_ld32(colS + 64 * h + 32, s1);
        maximum(s0, 2 * h);
        tmem_wait_ld();
        tmem_ld32(colS + 64 * (h ^ 1), s0);  // (at the end the first columns again)
        maximum(s1, 2 * h + 1);
      }
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
      // The reference moves when the maximum grew by more than 2^8 (until then p may reach 2^8).
      float m_old = -INFINITY;
      if (j > 0) {
        ok = max_wait(j - 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        m_old = lds32f(m_at);
      }
      const float m_new = top > m_old + 8.f ? top : m_old;
      sts32(m_at, __float_as_uint(m_new));
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::kBarMax + 4 * t + w4));
      if (m_new != m) {
        l *= ex2(m - m_new);
        m = m_new;
      }
      // O is rescaled when it did, or V's exponent fell, once the tile before is in it
      if (__any_sync(0xffffffffu, j > 0 && (m_new != m_old || e_new != e_old))) {
        ok = mbar_wait(bar(C::kBarVEmpty + (t ^ 1)), ((j - 1) >> 1) & 1, ctl);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const float a = (m_new != m_old ? ex2(m_old - m_new) : 1.f) * exp2i_or_zero(e_new - e_old);
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t ov[16];
          tmem_ld16(trow + C::kColO + 16 * c, ov);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * a);
          tmem_st16(trow + C::kColO + 16 * c, ov);
        }
      }
      // p = 2^(x * sc - m + 7) as fp16 pairs over S's columns (those of keys that are read by then)
      const float shift = (m == -INFINITY) ? 0.f : 7.f - m;
      const uint64_t sc2 = f2(sc, sc), shift2 = f2(shift, shift);
      uint64_t acc0 = f2(0.f, 0.f), acc1 = f2(0.f, 0.f);
      auto probabilities = [&](uint32_t (&v)[32], int c) {
        scores(v, c);
        uint32_t pk[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const uint64_t y =
              f2_fma(f2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), sc2, shift2);
          float y0, y1;
          f2_split(y, y0, y1);
          const float e0 = ex2(y0), e1 = ex2(y1);
          if (k & 1) acc1 = f2_add(acc1, f2(e0, e1)); else acc0 = f2_add(acc0, f2(e0, e1));
          pk[k] = pack_f16x2(e0, e1);
        }
        tmem_st16(colS + 16 * c, pk);
      };
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        tmem_wait_ld();
        tmem_ld32(colS + 64 * h + 32, s1);
        probabilities(s0, 2 * h);
        tmem_wait_ld();
        if (h == 0) tmem_ld32(colS + 64, s0);
        probabilities(s1, 2 * h + 1);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(C::kBarPFull + 2 * b + h));
      }
      float a0, a1, a2, a3;
      f2_split(acc0, a0, a1);
      f2_split(acc1, a2, a3);
      l += (a0 + a1) + (a2 + a3);
    }

    // ---- partial output O / l * 2^-E and log-sum-exp (log2 units; l carries 2^7) ----
    // The last tile's warpgroup has the final maximum; the scales' slots are free for the two sums.
    if (ok) {
      ok = mbar_wait(bar(C::kBarOFinal), 0, ctl) && (!warp_live || max_wait(nt - 1));
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
    }
    const float m_final = lds32f(m_at);
    const int e_final = static_cast<int>(lds32(sb + C::kExpOff + 8 * ((nt - 1) % 3)));
    if (m != m_final) l *= ex2(m - m_final);
    float* l_x = reinterpret_cast<float*>(smem + C::kKsOff);
    l_x[128 * t + r] = l;
    named_bar_sync(1, 256);
    l = l_x[r] + l_x[128 + r];
    const bool some = ok && warp_live && l != 0.f;
    const float inv_l = some ? 1.f / l : 0.f, unscale = exp2i(-e_final);
    const float lse = some ? (m_final + (log2f(l) - 7.f)) * 0.69314718055994531f : -INFINITY;
    // Rows are staged in K's slots (every product is done), to be written to global memory row by row:
    // each warpgroup half of the dims, 16-byte pieces XORed with the row.
    auto piece = [&](int row, int d) {  // of dims d .. d + 3
      return sb + C::kKOff + row * (D * 4) + (((d / 4) ^ (row & 7)) << 4);
    };
    if (warp_live) {
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {  // 16 dims
        const int d0 = t * (D / 2) + 16 * c;
        uint32_t ov[16];
        if (ok) {
          tmem_ld16(trow + C::kColO + d0, ov);
          tmem_wait_ld();
        }
#pragma unroll
        for (int q8 = 0; q8 < 2; ++q8) {
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            // INT4: column i of a chunk holds dim 0, 4, 2, 6, 1, 5, 3, 7
            const int dim = kBits == 4 ? ((i & 1) << 2 | (i & 2) | (i >> 2)) : i;
            f[dim] = some ? __uint_as_float(ov[8 * q8 + i]) * inv_l * unscale : 0.f;
          }
          sts128(piece(r, d0 + 8 * q8), __float_as_uint(f[0]), __float_as_uint(f[1]),
                 __float_as_uint(f[2]), __float_as_uint(f[3]));
          sts128(piece(r, d0 + 8 * q8 + 4), __float_as_uint(f[4]), __float_as_uint(f[5]),
                 __float_as_uint(f[6]), __float_as_uint(f[7]));
        }
      }
    }
    named_bar_sync(1, 256);
    const int out0 = 16 * warp;  // this warp writes rows out0 .. out0 + 15
    if (out0 < live || warp_live) {
      // Launched as a programmatic dependent of the kernel that reads the sequences' own keys: this grid
      // does not end before that one, so whoever waits for this one waits for both.
      asm volatile("griddepcontrol.wait;" ::: "memory");
      if (t == 0 && r < live) p.lse_part[split * rows + out_row(r)] = lse;
      const int orow = static_cast<int>(out_row(min(out0 + (lane & 15), live - 1)));
      constexpr int kLanes = D / 4;  // lanes of a row
      const int d = 4 * (lane % kLanes);
#pragma unroll 4
      for (int i = 0; i < 16; i += 32 / kLanes) {
        const int w = i + lane / kLanes;
        const int to = __shfl_sync(0xffffffffu, orow, w);
        const uint4 y = lds128(piece(out0 + w, d));
        if (out0 + w < live)
          *reinterpret_cast<uint4*>(p.o_part + (split * rows + to) * D + d) = y;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

}  // namespace fa
