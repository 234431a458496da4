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
// merges them: L = log sum_s exp(L_s), O = sum_s exp(L_s - L) O_s.  (For few rows or a short prefix the
// prefix goes through the split kernel as well, as one sequence of R rows: the launch decides.)
//
// fa_shared_prefix_kernel, one CTA per (KV head, block of rows, split of the prefix), 512 threads:
//   warps 0-3   softmax of S tile 0 (thread = query row = TMEM lane), warps 4-7 of S tile 1
//   warps 8-11  dequantisation: thread = key; K codes to fp16 (exact), V codes times their scale to
//               fp16, both into the swizzled layout the tensor core reads
//   warp 12     TMA producer: K and V code tiles of 128 keys, one box per page piece
//   warp 13     allocates TMEM and issues tcgen05.mma from one lane: S_t = Q_t K^T,
//               O_t += P_t V with P_t from TMEM
//   warp 14     the keys' scales, and the exponent E below;  warp 15 idles
// The two S tiles are two blocks of 128 query rows that share every K/V tile (kStream = false), or,
// when R <= 128, two interleaved streams of key tiles over one block of rows (kStream = true), merged
// as they are written; either way one tile's softmax runs while the tensor core works on the other.
//
// What bounds it: neither memory nor the tensor core but the chain of one tile - its softmax, then its
// P V and its next Q K^T, before which the next softmax cannot start (P lies over S).  With two
// tiles of 128 x 128 scores at D = 128, 4.6 thousand cycles a pair, of which a softmax warp computes 3.2 (exponentials 1.7,
// scaling and maximum 0.6) and the tensor core 2.05; 32768 keys x 64 sequences x 32 / 8 heads on 144 SMs
// 54 us, 640 TFLOP/s (B200).  Two things cost most on the way there: the unrolled code of all roles in the instruction
// caches, hence the rolled loops wherever registers allow, and operands of tcgen05.mma in vector registers,
// hence the converged MMA warp.
// A single accumulator with three buffers of S, which lets S run ahead of the softmax, is no faster: the
// registers and the converted tiles that it needs per row are twice as many.
//
// Number formats.  Q is scaled per row by a power of two and kept in fp16, which holds a bf16 row
// exactly (elements more than 2^29 below the row's largest lose bits, 2^25 for INT4).  Scores, maxima,
// sums, O and log-sum-exps are fp32; k_scale multiplies the fp32 scores, so QK^T has no rounding
// of its own.  P = 2^7 p (p <= 2^8 with the lazy maximum), v_scale * 2^E and its product with the code
// are rounded to fp16 (relative 2^-11 each, an eighth of the bf16 output's): the shift by 2^7 keeps
// weights down to 2^-31 of the maximum from vanishing, and the power E, lowered (with an exact rescale
// of O) when a larger v_scale arrives, keeps V below 2^15.
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

template <int D, int kBits, bool kStream>
struct SharedCfg {
  static constexpr int kThreads = 512;
  static constexpr int kRow = D * kBits / 8;       // bytes of one row of codes
  static constexpr int kAtom = 128 * 128;          // 128 rows x 128 bytes (64 fp16)
  static constexpr int kTile = 128 * D * 2;        // 128 rows of fp16
  static constexpr int kRawTile = 128 * kRow;
  static constexpr int kQTiles = kStream ? 1 : 2;
  // stages of code tiles: as many as fit beside two fp16 stages of K and V
  static constexpr int kRaw = (kStream || D == 64 || kBits == 4) ? 2 : 1;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQTiles * kTile;
  static constexpr int kVOff = kKOff + 2 * kTile;
  static constexpr int kRawKOff = kVOff + 2 * kTile;
  static constexpr int kRawVOff = kRawKOff + kRaw * kRawTile;
  static constexpr int kScaleOff = kRawVOff + kRaw * kRawTile;  // fp32 [2 tiles][k, v][128]
  static constexpr int kExpOff = kScaleOff + 2 * 2 * 512;       // int [2 tiles] V's exponent
  static constexpr int kBarOff = kExpOff + 16;
  static constexpr int kBarQ = 0;
  static constexpr int kBarRawKFull = 1;             // [kRaw]
  static constexpr int kBarRawVFull = kBarRawKFull + kRaw;
  static constexpr int kBarRawKEmpty = kBarRawVFull + kRaw;
  static constexpr int kBarRawVEmpty = kBarRawKEmpty + kRaw;
  static constexpr int kBarKFull = kBarRawVEmpty + kRaw;  // [2]
  static constexpr int kBarVFull = kBarKFull + 2;
  static constexpr int kBarKEmpty = kBarVFull + 2;
  static constexpr int kBarVEmpty = kBarKEmpty + 2;
  static constexpr int kBarScale = kBarVEmpty + 2;   // [2]
  static constexpr int kBarSFull = kBarScale + 2;    // [2]
  static constexpr int kBarPFull = kBarSFull + 2;    // [2 tiles][2 halves]
  static constexpr int kBarOFinal = kBarPFull + 4;   // [2]
  static constexpr int kBarDrain = kBarOFinal + 2;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr int kMiscOff = kBarOff + 8 * kNumBars;
  static constexpr int kSmemBytes = kMiscOff + 16;
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
  static constexpr uint32_t kTmemCols = 512;
  __host__ __device__ static constexpr uint32_t colS(int t) { return 128u * t; }
  __host__ __device__ static constexpr uint32_t colO(int t) { return 256u + uint32_t(D) * t; }
  // the launch's 512 x 128 registers: two softmax warpgroups, dequantisation, producer + MMA
  static constexpr uint32_t kRegsSoftmax = 192, kRegsDequant = 72, kRegsOther = 56;
  static constexpr int kLaunchRegs = 128;
  static_assert(2 * kRegsSoftmax + kRegsDequant + kRegsOther == 4 * kLaunchRegs, "register split");
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

// One key's row of codes (in the raw tile, swizzled by its TMA box) to fp16 in the layout of a
// tensor-core operand: 64-dim atoms of 128-byte rows, 16-byte chunk index XOR row % 8.  kScale:
// values times vs (an fp16 pair).  INT4: within each 8-dim chunk the dims stand in the order 0, 4,
// 2, 6, 1, 5, 3, 7 (that of the nibble extraction); the last four come out as 16 x the code,
// which vs_hi = vs / 16 or the other operand undoes.
template <int D, int kBits, bool kScale>
__device__ __forceinline__ void dequant_row(uint32_t raw, uint32_t dst, int r, uint32_t vs,
                                            uint32_t vs_hi) {
  constexpr int kRow = D * kBits / 8, kLoads = kBits / 2;  // 16-byte pieces of 64 dims' codes
#pragma unroll 1
  for (int atom = 0; atom < D / 64; ++atom) {
    const uint32_t row = dst + atom * (128 * 128) + r * 128;
    auto put = [&](int chunk, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
      if constexpr (kScale) {
        a = mul_f16x2(a, vs);
        b = mul_f16x2(b, vs);
        c = mul_f16x2(c, vs_hi);
        d = mul_f16x2(d, vs_hi);
      }
      sts128(row + ((chunk ^ (r & 7)) << 4), a, b, c, d);
    };
    uint4 x[kLoads];
#pragma unroll
    for (int c = 0; c < kLoads; ++c) x[c] = lds128(raw + swz<kRow>(r * kRow + 16 * (kLoads * atom + c)));
#pragma unroll
    for (int c = 0; c < kLoads; ++c) {
      const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
      if constexpr (kBits == 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t u = w[2 * h] ^ 0x80808080u, v = w[2 * h + 1] ^ 0x80808080u;
          put(2 * c + h, codes_to_f16x2(u, kSelB01), codes_to_f16x2(u, kSelB23),
              codes_to_f16x2(v, kSelB01), codes_to_f16x2(v, kSelB23));
        }
      } else {
#pragma unroll
        for (int h = 0; h < 4; ++h)
          put(4 * c + h, nib_lo_f16x2(w[h]), nib_lo_f16x2(w[h] >> 8), nib_hi16_f16x2(w[h]),
              nib_hi16_f16x2(w[h] >> 8));
      }
    }
  }
}

template <int D, int kBits, bool kStream>
__global__ void __launch_bounds__(512, 1)
    fa_shared_prefix_kernel(const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const SharedParams p) {
  using C = SharedCfg<D, kBits, kStream>;
  // the kernel of the sequences' own keys may start on the SMs that this grid leaves free
  asm volatile("griddepcontrol.launch_dependents;");
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
  const int row0 = rb * 256;
  const int live = min(kStream ? 128 : 256, p.R - row0);  // query rows of this CTA

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
    return;
  }
  const bool act1 = kStream ? nt > 1 : live > 128;  // S tile 1 has work

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kNumBars; ++i) {
      uint32_t count = 1;
      if (i == C::kBarQ) count = 256;
      if (i >= C::kBarPFull && i < C::kBarPFull + 4) count = 128;
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
  // What the warps read first is on its way before the barrier: the producer's and the scale warp's
  // page-table entries of the first tile, and the query rows (a warp fetches the 32 rows of its threads,
  // D / 8 lanes a row; streams: both warpgroups the same rows).
  const int box_t = min(128, 1 << p.page_shift), boxes = 128 / box_t;  // keys of a TMA box, boxes of a tile
  auto entry_at = [&](int j) -> int {  // of this lane's box, or of its 4 keys
    const int t = t_begin + 128 * j + lane * (warp == 12 ? box_t : 4);
    return j < nt && t < t_end && (warp != 12 || lane < boxes) ? __ldg(p.table + (t >> p.page_shift)) : 0;
  };
  int entry = 0;
  constexpr int kQLanes = D / 8, kQRows = 32 / kQLanes, kQSteps = 32 / kQRows;
  uint4 q_raw[kQSteps];
  const int R = (kStream || warp >= 8 ? 0 : (warp >> 2) * 128) + (threadIdx.x & 127);  // row of the CTA
  if (warp == 12 || warp == 14) {
    entry = entry_at(0);
  } else if (warp < 8) {
    const int mine = static_cast<int>(out_row(min(R, live - 1)));
#pragma unroll
    for (int i = 0; i < kQSteps; ++i) {
      const int row = i * kQRows + lane / kQLanes;
      const size_t from = __shfl_sync(0xffffffffu, mine, row);
      q_raw[i] = make_uint4(0, 0, 0, 0);
      if ((R & ~31) + row < live)
        q_raw[i] = __ldg(reinterpret_cast<const uint4*>(p.q + from * D) + lane % kQLanes);
    }
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
    setmaxnreg_dec<C::kRegsOther>();
    if (warp == 12) {
      // ================= TMA producer =================
      // lane i < boxes copies box i of each tile (a page, or 128 keys of a larger one); boxes past
      // the last key are skipped: the codes left there are finite and their scales count as 0
      const int pmask = (1 << p.page_shift) - 1;
      const uint32_t box_bytes = static_cast<uint32_t>(box_t) * C::kRow;
      const uint64_t pol = l2_evict_first_policy();
      int issued = 0;
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
      scales_at(0, entry, ks, vs);
      entry = entry_at(1);
      constexpr int kUnset = 1 << 20;
      int e0 = kUnset, e1 = kUnset;  // exponents of the accumulators of this tile and of the next
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
        const int e = min(e0, exponent_below(__uint_as_float(top), 8));
        e0 = kStream ? e1 : e;
        e1 = e;
        const float f = exp2i(e);
        const int slot = j & 1;
        const uint32_t dst = sb + C::kScaleOff + slot * 1024 + 16 * lane;
        // the slot is free once the products of tile j - 2 are done
        const bool ok = mbar_wait(bar(C::kBarVEmpty + slot), ((j >> 1) & 1) ^ 1, ctl);
        if (!__all_sync(0xffffffffu, ok)) break;
        sts128(dst, __float_as_uint(ks.x), __float_as_uint(ks.y), __float_as_uint(ks.z),
               __float_as_uint(ks.w));
        sts128(dst + 512, __float_as_uint(vs.x * f), __float_as_uint(vs.y * f),
               __float_as_uint(vs.z * f), __float_as_uint(vs.w * f));
        if (lane == 0) reinterpret_cast<volatile int*>(smem + C::kExpOff)[slot] = e;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kBarScale + slot));
        ks = ks_next;
        vs = vs_next;
      }
    } else if (warp == 13) {
      // ================= MMA issuer =================
      constexpr uint32_t idesc_qk = idesc_f16_f32(128, 128, false);
      constexpr uint32_t idesc_pv = idesc_f16_f32(128, D, true);
      // The whole warp runs the loop and one lane's instructions count: in code that one lane alone runs
      // the operands of each product went through vector registers, twice the time to issue it.
      const bool one = elect_one();
      // operand descriptors differ in the address field only (16-byte units, low word): one add each
      const uint64_t desc_k_major = smem_desc_sw128(0, 16, 1024);
      const uint64_t desc_v = smem_desc_sw128(0, C::kAtom, 1024);
      auto wait = [&](int b, int parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, ctl));
      };
      auto commit = [&](int b) { tc_commit_if(bar(b), one); };
      auto issue_qk = [&](int t, int slot) {
        const uint32_t qa = (sb + C::kQOff + (kStream ? 0 : t) * C::kTile) >> 4;
        const uint32_t kb = (sb + C::kKOff + slot * C::kTile) >> 4;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk / 4) * C::kAtom + (kk % 4) * 32) >> 4;
          umma_ss_if(tmem + C::colS(t), desc_k_major + (qa + off), desc_k_major + (kb + off), idesc_qk,
                     kk > 0 ? 1u : 0u, one);
        }
        commit(C::kBarSFull + t);
      };
      // O_t += P_t V; P_t arrives in two halves of 64 keys
      auto issue_pv = [&](int t, int slot, bool first, int phase) -> bool {
        const uint32_t vb = (sb + C::kVOff + slot * C::kTile) >> 4;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!wait(C::kBarPFull + 2 * t + half, phase)) return false;
          tc_fence_after();
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {
            const int kk = 4 * half + k4;
            umma_ts_if(tmem + C::colO(t), tmem + C::colS(t) + kk * 8, desc_v + (vb + kk * 128), idesc_pv,
                       (first && kk == 0) ? 0u : 1u, one);
          }
        }
        return true;
      };
      // tile j sits in slot j & 1 of K and V, in that slot's use number j >> 1
      auto k_wait = [&](int j) { return wait(C::kBarKFull + (j & 1), (j >> 1) & 1); };
      auto v_wait = [&](int j) { return wait(C::kBarVFull + (j & 1), (j >> 1) & 1); };
      bool ok = wait(C::kBarQ, 0);
      // (loops rolled: one copy of the issue code is what this warp's registers hold)
      if constexpr (kStream) {
#pragma unroll 1
        for (int j = -2; j < nt && ok; ++j) {
          const int t = j & 1;
          if (j >= 0) {
            ok = v_wait(j) && issue_pv(t, t, j < 2, (j >> 1) & 1);
            if (!ok) break;
            commit(C::kBarVEmpty + t);
            if (j + 2 >= nt) commit(C::kBarOFinal + t);
          }
          if (j + 2 < nt) {
            if (!(ok = k_wait(j + 2))) break;
            tc_fence_after();
            issue_qk(t, t);
            commit(C::kBarKEmpty + t);
          }
        }
      } else {
        const int last = act1 ? 1 : 0;
#pragma unroll 1
        for (int j = -1; j < nt && ok; ++j) {
          if (j >= 0 && !(ok = v_wait(j))) break;
#pragma unroll 1
          for (int t = 0; t <= last && ok; ++t) {
            if (j >= 0) {
              if (!(ok = issue_pv(t, j & 1, j == 0, j & 1))) break;
              if (t == last) commit(C::kBarVEmpty + (j & 1));
              if (j + 1 == nt) commit(C::kBarOFinal + t);
            }
            if (j + 1 < nt) {
              if (t == 0 && !(ok = k_wait(j + 1))) break;
              tc_fence_after();
              issue_qk(t, (j + 1) & 1);
              if (t == last) commit(C::kBarKEmpty + ((j + 1) & 1));
            }
          }
        }
      }
      // Drain: every MMA this warp issued has completed before TMEM is released.
      commit(C::kBarDrain);
      volatile int zero = 0;
      const WaitCtl drain_ctl{&zero, p.timeout_ns};
      mbar_wait(bar(C::kBarDrain), 0, drain_ctl);
    }
  } else if (warp >= 8) {
    setmaxnreg_dec<C::kRegsDequant>();
    // ================= dequantisation: thread r = key r of each tile =================
    const int r = threadIdx.x & 127;
    for (int j = 0; j < nt; ++j) {
      const int s = j % C::kRaw, ph = (j / C::kRaw) & 1, slot = j & 1, use = (j >> 1) & 1;
      bool ok = mbar_wait(bar(C::kBarKEmpty + slot), use ^ 1, ctl) &&
                mbar_wait(bar(C::kBarRawKFull + s), ph, ctl);
      if (!__all_sync(0xffffffffu, ok)) break;
      dequant_row<D, kBits, false>(sb + C::kRawKOff + s * C::kRawTile,
                                   sb + C::kKOff + slot * C::kTile, r, 0u, 0u);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(C::kBarRawKEmpty + s));
        mbar_arrive(bar(C::kBarKFull + slot));
      }
      // (the scales' slot is written after V's is free)
      ok = mbar_wait(bar(C::kBarScale + slot), use, ctl) &&
           mbar_wait(bar(C::kBarRawVFull + s), ph, ctl);
      if (!__all_sync(0xffffffffu, ok)) break;
      const float vs = lds32f(sb + C::kScaleOff + slot * 1024 + 512 + 4 * r);
      dequant_row<D, kBits, true>(sb + C::kRawVOff + s * C::kRawTile,
                                  sb + C::kVOff + slot * C::kTile, r, pack_f16x2(vs, vs),
                                  kBits == 4 ? pack_f16x2(vs * 0.0625f, vs * 0.0625f)
                                             : pack_f16x2(vs, vs));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(C::kBarRawVEmpty + s));
        mbar_arrive(bar(C::kBarVFull + slot));
      }
    }
  } else {
    setmaxnreg_inc<C::kRegsSoftmax>();
    // ================= Q, softmax, epilogue: thread r = query row r of S tile t =================
    const int t = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const uint32_t colS = t ? C::colS(1) : C::colS(0);
    const uint32_t colO = t ? C::colO(1) : C::colO(0);
    const bool warp_live = (R & ~31) < live;  // a warp of padding rows only keeps the barriers
    const int first = kStream ? t : 0, step = kStream ? 2 : 1;

    float sc = 0.f;  // of row R: score units of log2, undoing the row's power of two
#pragma unroll 1  // (short code: it runs once, from a cold instruction cache)
    for (int i0 = 0; i0 < kQSteps; i0 += 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 x = q_raw[i];
        if constexpr (kQSteps > 8) q_raw[i] = q_raw[i + 8];
        const int row = (r & ~31) + (i0 + i) * kQRows + lane / kQLanes, c = lane % kQLanes;  // of the tile
        const uint32_t kAbs = 0x7fff7fffu;
        uint32_t am = __vmaxu2(__vmaxu2(x.x & kAbs, x.y & kAbs), __vmaxu2(x.z & kAbs, x.w & kAbs));
#pragma unroll
        for (int o = 1; o < kQLanes; o <<= 1) am = __vmaxu2(am, __shfl_xor_sync(0xffffffffu, am, o));
        const int eq = exponent_below(__uint_as_float(max(am & 0xffffu, am >> 16) << 16), 15);
        // (not 0: a masked score is -infinity times this)
        const float sc_i = __shfl_sync(0xffffffffu, fmaxf(p.scale_log2 * exp2i(-eq), 0x1p-126f),
                                       lane % kQRows * kQLanes);
        if (lane / kQRows == i0 + i) sc = sc_i;
        if (kStream && (i & 1) != t) continue;  // each warpgroup lays out half of the rows
        const float qs = exp2i(eq);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
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
        sts128(sb + C::kQOff + (kStream ? 0 : t) * C::kTile + (c >> 3) * C::kAtom + row * 128 +
                   (((c & 7) ^ (row & 7)) << 4), h[0], h[1], h[2], h[3]);
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(bar(C::kBarQ));

    float m = -INFINITY, l = 0.f;
    constexpr int kUnset = 1 << 20;
    int E = kUnset, n = 0;
    for (int j = first; j < (t == 0 || act1 ? nt : 0); j += step, ++n) {
      bool ok = mbar_wait(bar(C::kBarSFull + t), n & 1, ctl);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      if (!warp_live) {  // whatever P holds for padding rows stays in those rows
        mbar_arrive(bar(C::kBarPFull + 2 * t));
        mbar_arrive(bar(C::kBarPFull + 2 * t + 1));
        continue;
      }
      uint32_t sv[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(trow + colS + 32 * c, sv[c]);
      ok = mbar_wait(bar(C::kBarScale + (j & 1)), (j >> 1) & 1, ctl);
      if (!__all_sync(0xffffffffu, ok)) break;
      const int e_new = static_cast<int>(lds32(sb + C::kExpOff + 4 * (j & 1)));
      tmem_wait_ld();
      // raw scores times k_scale (the row's common factor sc joins in the exponent), and their maximum
      const uint32_t ring = sb + C::kScaleOff + (j & 1) * 1024;
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int q4 = 0; q4 < 8; ++q4) {
          const uint4 k4 = lds128(ring + 128 * c + 16 * q4);
          const uint64_t a = f2_mul(f2(__uint_as_float(sv[c][4 * q4]), __uint_as_float(sv[c][4 * q4 + 1])),
                                    f2(__uint_as_float(k4.x), __uint_as_float(k4.y)));
          const uint64_t b = f2_mul(f2(__uint_as_float(sv[c][4 * q4 + 2]), __uint_as_float(sv[c][4 * q4 + 3])),
                                    f2(__uint_as_float(k4.z), __uint_as_float(k4.w)));
          float a0, a1, b0, b1;
          f2_split(a, a0, a1);
          f2_split(b, b0, b1);
          sv[c][4 * q4] = __float_as_uint(a0);
          sv[c][4 * q4 + 1] = __float_as_uint(a1);
          sv[c][4 * q4 + 2] = __float_as_uint(b0);
          sv[c][4 * q4 + 3] = __float_as_uint(b1);
          mx[2 * (q4 & 1)] = fmax3(mx[2 * (q4 & 1)], a0, a1);
          mx[2 * (q4 & 1) + 1] = fmax3(mx[2 * (q4 & 1) + 1], b0, b1);
        }
      float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      const int limit = t_end - (t_begin + 128 * j);
      if (limit < 128) {
        top = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            if (32 * c + k >= limit) sv[c][k] = __float_as_uint(-INFINITY);
            top = fmaxf(top, __uint_as_float(sv[c][k]));
          }
      }
      const float m_new = fmaxf(m, top * sc);
      // O is rescaled when the maximum grew by more than 2^8 (until then the old one stays the
      // reference and p may reach 2^8) or V's exponent fell
      float alpha = 1.f;
      bool resc = false;
      if (n == 0) {
        m = m_new;
      } else {
        if (m_new > m + 8.f) {
          resc = true;
          alpha = ex2(m - m_new);
          m = m_new;
        }
        resc = resc || e_new != E;
      }
      if (__any_sync(0xffffffffu, resc)) {
        const float a = alpha * exp2i_or_zero(e_new - E);
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t ov[16];
          tmem_ld16(trow + colO + 16 * c, ov);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * a);
          tmem_st16(trow + colO + 16 * c, ov);
        }
      }
      E = e_new;
      // p = 2^(x * sc - m + 7) as fp16 pairs over S's columns, one half of the keys at a time
      const float shift = (m == -INFINITY) ? 0.f : 7.f - m;
      const uint64_t sc2 = f2(sc, sc), shift2 = f2(shift, shift);
      uint64_t acc0 = f2(0.f, 0.f), acc1 = f2(0.f, 0.f);
#pragma unroll
      for (int piece = 0; piece < 4; ++piece) {  // 32 keys
        uint32_t pk[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const uint64_t x = f2_fma(f2(__uint_as_float(sv[piece][2 * k]),
                                       __uint_as_float(sv[piece][2 * k + 1])),
                                    sc2, shift2);
          float x0, x1;
          f2_split(x, x0, x1);
          const float a = ex2(x0), b = ex2(x1);
          if (k & 1) acc1 = f2_add(acc1, f2(a, b)); else acc0 = f2_add(acc0, f2(a, b));
          pk[k] = pack_f16x2(a, b);
        }
        tmem_st16(trow + colS + 16 * piece, pk);
        if (piece & 1) {
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(bar(C::kBarPFull + 2 * t + (piece >> 1)));
        }
      }
      float a0, a1, a2, a3;
      f2_split(acc0, a0, a1);
      f2_split(acc1, a2, a3);
      l = l * alpha + ((a0 + a1) + (a2 + a3));
    }

    // ---- partial output O / l * 2^-E and log-sum-exp (log2 units; l carries 2^7) ----
    bool have = false;
    if (n > 0) {
      const bool ok = mbar_wait(bar(C::kBarOFinal + t), 0, ctl);
      have = __all_sync(0xffffffffu, ok);
      tc_fence_after();
    }
    const bool some = have && warp_live && l != 0.f;
    const float inv_l = some ? 1.f / l : 0.f;
    const float unscale = E == kUnset ? 0.f : exp2i(-E);
    const float lse2 = some ? m + (log2f(l) - 7.f) : -INFINITY;
    // Rows are staged in shared memory, to be written to global memory row by row, and so that both
    // streams' rows can be merged.  What is free by now: tile 0's products of QK^T and its own of PV
    // are done (K's slots), tile 1's last of all (V's slots); streams each have a slot of K and of V
    // to themselves.  Half of a row's dims in each of two areas, 16-byte pieces XORed with the row.
    const uint32_t areas = kStream ? C::kVOff - C::kKOff : C::kTile;  // from the first to the second
    const uint32_t area0 = sb + (kStream ? C::kKOff + t * C::kTile : t ? C::kVOff : C::kKOff);
    auto piece = [&](uint32_t base, int row, int d) {  // of dims d .. d + 3
      constexpr int kHalf = D / 2;
      return base + (d < kHalf ? 0u : areas) + row * (kHalf * 4) +
             ((((d % kHalf) / 4) ^ (row & 7)) << 4);
    };
    if (have && warp_live) {
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t ov[32];
        tmem_ld32(trow + colO + 32 * c, ov);
        tmem_wait_ld();
#pragma unroll
        for (int q8 = 0; q8 < 4; ++q8) {
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            // INT4: column i of a chunk holds dim 0, 4, 2, 6, 1, 5, 3, 7
            const int dim = kBits == 4 ? ((i & 1) << 2 | (i & 2) | (i >> 2)) : i;
            f[dim] = some ? __uint_as_float(ov[8 * q8 + i]) * inv_l * unscale : 0.f;
          }
          const int d = 32 * c + 8 * q8;
          sts128(piece(area0, r, d), __float_as_uint(f[0]), __float_as_uint(f[1]),
                 __float_as_uint(f[2]), __float_as_uint(f[3]));
          sts128(piece(area0, r, d + 4), __float_as_uint(f[4]), __float_as_uint(f[5]),
                 __float_as_uint(f[6]), __float_as_uint(f[7]));
        }
      }
    }
    // rows that this warp writes: its own or (streams, 8 warps for 128 rows) 16
    constexpr int kOut = kStream ? 16 : 32;
    const int out0 = kStream ? 16 * warp : R & ~31;
    const int tile0 = kStream ? out0 : r & ~31;  // ... counted in the tile
    float w0 = 1.f, w1 = 0.f, lse_row = lse2;
    if constexpr (kStream) {
      // (in the scales' slot that this stream's tiles used)
      float* lse_x = reinterpret_cast<float*>(smem + C::kScaleOff);
      lse_x[256 * t + r] = lse2;
      named_bar_sync(1, 256);
      const float a = lse_x[out0 + (lane & 15)], b = lse_x[256 + out0 + (lane & 15)];
      const float top = fmaxf(a, b);
      w0 = a == -INFINITY ? 0.f : ex2(a - top);
      w1 = b == -INFINITY ? 0.f : ex2(b - top);
      const float sum = w0 + w1;
      lse_row = sum == 0.f ? -INFINITY : top + log2f(sum);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      // -1: a stream without keys, which has staged nothing. A weight of 0 still counts: its stream may hold a NaN
      w0 = a == -INFINITY ? -1.f : w0 * inv;
      w1 = b == -INFINITY ? -1.f : w1 * inv;
    } else {
      __syncwarp();
    }
    if (out0 < live) {
      const int mine = out0 + (lane & (kOut - 1));
      const int orow = static_cast<int>(out_row(min(mine, live - 1)));
      if (lane < kOut && mine < live) p.lse_part[split * rows + orow] = lse_row * 0.69314718055994531f;
      constexpr int kLanes = D / 4;  // lanes of a row
      const int d = 4 * (lane % kLanes);
      const uint32_t from = kStream ? sb + C::kKOff : area0;
#pragma unroll 4
      for (int i = 0; i < kOut; i += 32 / kLanes) {
        const int w = i + lane / kLanes;
        const int to = __shfl_sync(0xffffffffu, orow, w);
        uint4 y = lds128(piece(from, tile0 + w, d));
        if constexpr (kStream) {
          const float u0 = __shfl_sync(0xffffffffu, w0, w), u1 = __shfl_sync(0xffffffffu, w1, w);
          const uint4 z = lds128(piece(from + C::kTile, tile0 + w, d));
          auto merge = [&](uint32_t a, uint32_t b) {
            return __float_as_uint((u0 < 0.f ? 0.f : u0 * __uint_as_float(a)) +
                                   (u1 < 0.f ? 0.f : u1 * __uint_as_float(b)));
          };
          y = make_uint4(merge(y.x, z.x), merge(y.y, z.y), merge(y.z, z.z), merge(y.w, z.w));
        }
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
