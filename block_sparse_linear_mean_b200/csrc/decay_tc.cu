// Linear attention with a decay for each head on the tensor cores (bf16
// operands, fp32 accumulators; decay_kernels.cu has the formulas and roles).
//
// Chunks of 128 tokens.  Per chunk, with S the state at its entering side:
//   X = a b^T                                    (K-major x K-major)
//   P = X o D, D_ij = w_in decay^(i-j)           (registers, bf16 into TMEM)
//   Z = a bf16(S),  O = P c                      (TMEM A for P)
//   out_i = O_i + w_st decay^(i+1-e) Z_i         (registers, fp32)
//   S <- decay^n S + (w b)^T c                   (accumulates in TMEM)
//
// Roundings to bf16 beside the inputs' own: P, S as operand of Z, and w b:
// one each per term of a bf16 result.  The state that is handed on (to the
// next segment, to the caller) does not come from there: decay_sums_tc
// splits w b into three bf16 parts (hi + lo + lo2, 24 bits together), so
// its sums have fp32 accuracy.
#include <algorithm>

#include "common.cuh"
#include "decay.cuh"
#include "tc_common.cuh"

namespace sla {

namespace {

constexpr int kC = 128;            // tokens per chunk
constexpr int kThreads = 320;      // 8 worker warps, loader, issuer

__device__ __forceinline__ uint8_t* align1k(uint8_t* p) {
  const uint32_t a = smem_u32(p);
  return p + (((a + 1023u) & ~1023u) - a);
}

// All waits of a CTA: bounded, and given up as soon as another warp has.
struct Waiter {
  int32_t* status;
  volatile int* abort_flag;
  long long limit;
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    const long long t0 = clock64();
    for (uint32_t it = 0;; ++it) {
      if (mbar_try_wait(bar, parity)) return true;
      if ((it & 63u) == 63u) {
        if (*abort_flag) return false;
        if (clock64() - t0 > limit) {
          *abort_flag = 1;
          atomicExch(status, 5 /* SLA_ERR_TIMEOUT */);
          return false;
        }
      }
    }
  }
};

// After a wait that gave up: the copies and products in flight end within
// this time; nothing of the CTA's memory is given back before.
__device__ __forceinline__ void drain(bool ok) {
  if (!ok) {
    const long long t0 = clock64();
    while (clock64() - t0 < 2000000) __nanosleep(1000);
  }
}

// Token rows [t0 + 128 n, + nc) of a segment of n_tok real tokens at t0; the
// walk goes over n from the entering side.
struct Chunks {
  int t0, tokens, count;
  bool reverse;
  __device__ __forceinline__ int at(int n) const { return reverse ? count - 1 - n : n; }
  __device__ __forceinline__ int row(int n) const { return t0 + at(n) * kC; }
  __device__ __forceinline__ int size(int n) const { return min(kC, tokens - at(n) * kC); }
};

// [128][D] tile as D / 64 swizzled halves of 16 KB each.
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, int row, int bh,
                                          uint32_t bar) {
#pragma unroll
  for (int h = 0; h < D / 64; ++h) tma_load_3d(dst + h * 16384, map, h * 64, row, bh, bar);
}

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// ---------------------------------------------------------------------------
// Segment sums: sums[bh][seg] = w_sum sum_i decay^(n-1-i+e) b_i^T c_i.
//
// Weights count from the segment's far end, so the accumulator is never
// scaled and the chunks' order is free: from the leaving side to the entering
// one, so that what the output kernel reads first was read last and is still
// in L2.  Eight warps turn a b tile into its three weighted parts (hi in
// place), the issuer multiplies.  With d = 64 hi and lo are stacked to the 128
// rows of one product and lo2 goes to an accumulator of its own.
struct SumsRole {
  float w_sum;
  int e;
  int reverse;
};

template <int D>
struct SumsSmem {
  static constexpr uint32_t tile = 128 * D * 2;
  static constexpr uint32_t stage = 2 * tile;          // b, c
  static constexpr uint32_t off_lo = 2 * stage;        // d = 128: lo, lo2; d = 64: lo2, hi, lo
  static constexpr uint32_t parts = D == 128 ? 2 : 3;
  static constexpr uint32_t off_bar = off_lo + parts * tile;
  static constexpr uint32_t total = off_bar + 128 + 512 + 1024;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    decay_sums_tc(const __grid_constant__ CUtensorMap mb0, const __grid_constant__ CUtensorMap mc0,
                  const __grid_constant__ CUtensorMap mb1, const __grid_constant__ CUtensorMap mc1,
                  const float* __restrict__ log_decay, const int32_t* __restrict__ lens,
                  float* __restrict__ sums0, float* __restrict__ sums1, DecayPlan P, SumsRole R0,
                  SumsRole R1, int32_t* status, int32_t* zero, long long limit, int withhold) {
  using L = SumsSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = align1k(smem_raw);
  const uint32_t sb = smem_u32(base);
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + L::off_bar);
  const uint32_t b_full = smem_u32(bars), b_empty = smem_u32(bars + 2), b_ready = smem_u32(bars + 4),
                 b_done = smem_u32(bars + 5);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 6);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 7);
  float* pw = reinterpret_cast<float*>(base + L::off_bar + 128);  // decay^k, k < 128
  const int tid = threadIdx.x, warp = tid / 32;
  const int seg = blockIdx.x, bh = blockIdx.y;
  const bool second = blockIdx.z != 0;
  const SumsRole R = second ? R1 : R0;
  const CUtensorMap* mb = second ? &mb1 : &mb0;
  const CUtensorMap* mc = second ? &mc1 : &mc0;
  if (zero && tid == 0 && seg == 0 && bh == 0 && !second) *zero = 0;
  const double l2 = decay_log2(log_decay[bh % P.H]);
  const int n = segment_tokens(P, lens, bh / P.H, seg);
  const Chunks ch{seg * P.seg_len, n, (n + kC - 1) / kC, R.reverse == 0};  // against the direction
  if (tid == 0) {
    mbar_init(b_full, 1);
    mbar_init(b_full + 8, 1);
    mbar_init(b_empty, 1);
    mbar_init(b_empty + 8, 1);
    mbar_init(b_ready, 8);
    mbar_init(b_done, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid < kC) pw[tid] = decay_power(l2, tid);
  if (warp == 9) tmem_alloc(smem_u32(tslot), 128);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const Waiter wait{status, abort_flag, limit};
  bool ok = true;

  if (warp == 8) {
    if (tid % 32 == 0) {
      for (int i = 0; ok && i < ch.count; ++i) {
        const int s = i & 1;
        if (i >= 2) ok = wait(b_empty + 8 * s, ((i >> 1) & 1) ^ 1);
        if (!ok) break;
        mbar_expect_tx(b_full + 8 * s, L::stage);
        if (!(withhold && i == 0 && seg == 0 && bh == 0))
          load_tile<D>(sb + s * L::stage, mb, ch.row(i), bh, b_full + 8 * s);
        load_tile<D>(sb + s * L::stage + L::tile, mc, ch.row(i), bh, b_full + 8 * s);
      }
    }
  } else if (warp == 9) {
    if (tid % 32 == 0) {
      constexpr uint32_t idesc = idesc_bf16(128, D, 1, 1);
      for (int i = 0; ok && i < ch.count; ++i) {
        const int s = i & 1;
        ok = wait(b_full + 8 * s, (i >> 1) & 1) && wait(b_ready, i & 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t dc = sdesc(sb + s * L::stage + L::tile, 16384, 1024);
        const uint64_t dh = sdesc(D == 128 ? sb + s * L::stage : sb + L::off_lo + L::tile, 16384, 1024);
        const uint64_t d2 = sdesc(sb + L::off_lo, 16384, 1024);
        const uint64_t d3 = sdesc(sb + L::off_lo + L::tile, 16384, 1024);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint64_t c = sdesc_add(dc, kk * 2048);
          const uint32_t acc = (i > 0 || kk > 0) ? 1u : 0u;
          tc_mma(tmem, sdesc_add(dh, kk * 2048), c, idesc, acc);
          if constexpr (D == 128) {
            tc_mma(tmem, sdesc_add(d2, kk * 2048), c, idesc, 1u);
            tc_mma(tmem, sdesc_add(d3, kk * 2048), c, idesc, 1u);
          } else {
            // rows 64 .. 127 take the tile behind lo2 (hi again); that half of
            // this accumulator is not read
            tc_mma(tmem + 64, sdesc_add(d2, kk * 2048), c, idesc, acc);
          }
        }
        tc_commit(b_done);
        tc_commit(b_empty + 8 * s);
      }
    }
  } else {
    for (int i = 0; ok && i < ch.count; ++i) {
      const int s = i & 1, nc = ch.size(i);
      // tokens left behind row r of the chunk, toward the leaving side
      const int row0 = ch.at(i) * kC;
      ok = __all_sync(0xffffffffu, wait(b_full + 8 * s, (i >> 1) & 1));
      if (ok && i > 0) ok = __all_sync(0xffffffffu, wait(b_done, (i - 1) & 1));
      if (!ok) break;
      const int r = tid & 127;
      // distance of the chunk's nearest real token from the leaving side
      const int near = R.reverse ? row0 : n - row0 - nc;
      const float far_w = R.w_sum * decay_power(l2, near + R.e);
      const float w = r < nc ? far_w * pw[R.reverse ? r : nc - 1 - r] : 0.f;
      uint8_t* bt = base + s * L::stage;
      uint8_t* hi_t = D == 128 ? bt : base + L::off_lo + L::tile;
      uint8_t* lo_t = base + L::off_lo + (D == 128 ? 0 : 2 * L::tile);
      uint8_t* l2_t = base + L::off_lo + (D == 128 ? L::tile : 0);
      constexpr int U = D / 16;  // 16-byte units per thread: half a row
#pragma unroll 4
      for (int x = 0; x < U; ++x) {
        const int u = (tid >> 7) * U + x;
        const uint32_t off = (u >> 3) * 16384 + sw128(r, u & 7);
        uint4 q = *reinterpret_cast<const uint4*>(bt + off);
        if (r >= nc) {
          q = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(bt + L::tile + off) = q;  // c: nothing may stand behind a weight of 0
        }
        uint32_t in[4] = {q.x, q.y, q.z, q.w}, h[4], l[4], m[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float a = w * lo_bf16(in[y]), b = w * hi_bf16(in[y]);
          h[y] = pack_bf16x2(a, b);
          const float a1 = a - lo_bf16(h[y]), b1 = b - hi_bf16(h[y]);
          l[y] = pack_bf16x2(a1, b1);
          m[y] = pack_bf16x2(a1 - lo_bf16(l[y]), b1 - hi_bf16(l[y]));
        }
        *reinterpret_cast<uint4*>(hi_t + off) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(lo_t + off) = make_uint4(l[0], l[1], l[2], l[3]);
        *reinterpret_cast<uint4*>(l2_t + off) = make_uint4(m[0], m[1], m[2], m[3]);
      }
      fence_async_smem();
      __syncwarp();
      if (tid % 32 == 0) mbar_arrive(b_ready);
    }
    if (ok && ch.count > 0) ok = __all_sync(0xffffffffu, wait(b_done, (ch.count - 1) & 1));
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  ok = __syncthreads_and(ok && !*abort_flag);
  // the accumulator, row = channel of b, to global memory
  float* dst = (second ? sums1 : sums0) + (i64(bh) * P.segs + seg) * D * D;
  if (ok && ch.count > 0) {
    tc_fence_after();
    const uint32_t lane = static_cast<uint32_t>((warp & 3) * 32) << 16;
    if constexpr (D == 128) {
      if (warp < 8) {
        const int row = tid & 127, c0 = (warp >> 2) * 64;
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          float v[32];
          tmem_ld32(tmem + lane + c0 + c, v);
          tmem_wait_ld();
          reg_fence<32>(v);
#pragma unroll
          for (int x = 0; x < 32; x += 4)
            *reinterpret_cast<float4*>(dst + row * D + c0 + c + x) = make_float4(v[x], v[x + 1], v[x + 2], v[x + 3]);
        }
      }
    } else {
      // rows 64 .. 127 hold the lo parts: through shared memory to the warps
      // of rows 0 .. 63 (stage 0 is free)
      float* xch = reinterpret_cast<float*>(base);
      if (warp == 2 || warp == 3) {
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          float v[32];
          tmem_ld32(tmem + lane + c, v);
          tmem_wait_ld();
          reg_fence<32>(v);
#pragma unroll
          for (int x = 0; x < 32; ++x) xch[(c + x) * 64 + (tid & 63)] = v[x];
        }
      }
      __syncthreads();
      if (warp < 2) {
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          float v[32], m[32];
          tmem_ld32(tmem + lane + c, v);
          tmem_ld32(tmem + lane + 64 + c, m);
          tmem_wait_ld();
          reg_fence<32>(v);
          reg_fence<32>(m);
#pragma unroll
          for (int x = 0; x < 32; ++x) v[x] += xch[(c + x) * 64 + tid] + m[x];
#pragma unroll
          for (int x = 0; x < 32; x += 4)
            *reinterpret_cast<float4*>(dst + tid * D + c + x) = make_float4(v[x], v[x + 1], v[x + 2], v[x + 3]);
        }
      }
    }
  } else if (ok) {
    for (int u = tid; u < D * D; u += kThreads) dst[u] = 0.f;  // no token
  }
  drain(ok);
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 128);
  }
}

// ---------------------------------------------------------------------------
// Outputs of a segment, chunk by chunk.  Warps 0-3 (row = thread) turn X into
// P and write the results; warps 4-7 take the state from TMEM to its bf16
// copy and weight the b tile in place; warp 8 loads, warp 9 issues.
template <int D>
struct OutSmem {
  static constexpr uint32_t tile = 128 * D * 2;
  static constexpr uint32_t stage = 3 * tile;              // a, b, c
  static constexpr uint32_t off_s = 2 * stage;             // bf16 state, [d][d]
  static constexpr uint32_t s_bytes = D * D * 2;
  static constexpr uint32_t off_bar = off_s + s_bytes;
  static constexpr uint32_t off_tab = off_bar + 128;       // decay^k, k <= 128
  static constexpr uint32_t total = off_tab + 130 * 4 + 1024;
};

template <int D, bool REV>
__global__ void __launch_bounds__(kThreads, 1)
    decay_out_tc(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                 const __grid_constant__ CUtensorMap mc, const float* __restrict__ log_decay,
                 const int32_t* __restrict__ lens, const float* __restrict__ starts, i64 start_stride,
                 __nv_bfloat16* __restrict__ out, DecayPlan P, DecayRole R, int32_t* status,
                 int32_t* zero, long long limit, int withhold) {
  using L = OutSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = align1k(smem_raw);
  const uint32_t sb = smem_u32(base);
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + L::off_bar);
  const uint32_t b_full = smem_u32(bars), b_empty = smem_u32(bars + 2);
  const uint32_t b_x = smem_u32(bars + 4);    // X in TMEM
  const uint32_t b_p = smem_u32(bars + 5);    // P in TMEM
  const uint32_t b_o = smem_u32(bars + 6);    // O and Z in TMEM
  const uint32_t b_free = smem_u32(bars + 7); // O and Z read
  const uint32_t b_s = smem_u32(bars + 8);    // state updated
  const uint32_t b_sr = smem_u32(bars + 9);   // bf16 state written, accumulator scaled
  const uint32_t b_h = smem_u32(bars + 10);   // b weighted
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 11);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 12);
  float* pw = reinterpret_cast<float*>(base + L::off_tab);
  const int tid = threadIdx.x, warp = tid / 32, quad = warp & 3;
  const int seg = blockIdx.x, bh = blockIdx.y;
  if (zero && tid == 0 && seg == 0 && bh == 0) *zero = 0;
  const double l2 = decay_log2(log_decay[bh % P.H]);
  const int n = segment_tokens(P, lens, bh / P.H, seg);
  const Chunks ch{seg * P.seg_len, n, (n + kC - 1) / kC, REV};
  if (tid == 0) {
    mbar_init(b_full, 1);
    mbar_init(b_full + 8, 1);
    mbar_init(b_empty, 1);
    mbar_init(b_empty + 8, 1);
    mbar_init(b_x, 1);
    mbar_init(b_p, 4);
    mbar_init(b_o, 1);
    mbar_init(b_free, 4);
    mbar_init(b_s, 1);
    mbar_init(b_sr, 4);
    mbar_init(b_h, 4);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid <= kC) pw[tid] = decay_power(l2, tid);
  if (warp == 9) tmem_alloc(smem_u32(tslot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tX = *tslot, tO = tX + 128, tZ = tO + D, tS = tZ + D;  // P over X
  const Waiter wait{status, abort_flag, limit};
  const unsigned all = 0xffffffffu;
  bool ok = true;

  if (warp == 8) {
    if (tid % 32 == 0) {
      for (int i = 0; ok && i < ch.count; ++i) {
        const int s = i & 1;
        if (i >= 2) ok = wait(b_empty + 8 * s, ((i >> 1) & 1) ^ 1);
        if (!ok) break;
        const uint32_t st = sb + s * L::stage, bar = b_full + 8 * s;
        mbar_expect_tx(bar, L::stage);
        if (!(withhold && i == 0 && seg == 0 && bh == 0)) load_tile<D>(st, &ma, ch.row(i), bh, bar);
        load_tile<D>(st + L::tile, &mb, ch.row(i), bh, bar);
        load_tile<D>(st + 2 * L::tile, &mc, ch.row(i), bh, bar);
      }
    }
  } else if (warp == 9) {
    if (tid % 32 == 0) {
      constexpr uint32_t id_x = idesc_bf16(128, 128, 0, 0), id_o = idesc_bf16(128, D, 0, 1),
                         id_s = idesc_bf16(128, D, 1, 1);
      const uint64_t ds = sdesc(sb + L::off_s, D * 128, 1024);
      for (int i = 0; i < ch.count; ++i) {
        const int s = i & 1;
        const uint32_t st = sb + s * L::stage;
        const uint64_t da = sdesc(st, 16, 1024), db = sdesc(st + L::tile, 16, 1024);
        const uint64_t dbt = sdesc(st + L::tile, 16384, 1024), dc = sdesc(st + 2 * L::tile, 16384, 1024);
        if (!(ok = wait(b_full + 8 * s, (i >> 1) & 1))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          tc_mma(tX, sdesc_add(da, off), sdesc_add(db, off), id_x, kk > 0);
        }
        tc_commit(b_x);
        if (!(ok = wait(b_sr, i & 1))) break;
        if (i > 0 && !(ok = wait(b_free, (i - 1) & 1))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma(tZ, sdesc_add(da, (kk >> 2) * 16384 + (kk & 3) * 32), sdesc_add(ds, kk * 2048), id_o, kk > 0);
        if (!(ok = wait(b_h, i & 1))) break;
        tc_fence_after();
        if (i + 1 < ch.count) {  // (behind the last chunk nobody reads the state)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc_mma(tS, sdesc_add(dbt, kk * 2048), sdesc_add(dc, kk * 2048), id_s, 1u);
          tc_commit(b_s);
        }
        if (!(ok = wait(b_p, i & 1))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          tc_mma_ts(tO, tX + kk * 8, sdesc_add(dc, kk * 2048), id_o, kk > 0);
        tc_commit(b_o);
        tc_commit(b_empty + 8 * s);
      }
    }
  } else if (warp < 4) {
    // ------------------------------------------------ P and the results
    const int r = tid;
    const uint32_t lane = static_cast<uint32_t>(quad * 32) << 16;
    for (int i = 0; ok && i < ch.count; ++i) {
      const int nc = ch.size(i);
      if (!(ok = __all_sync(all, wait(b_x, i & 1)))) break;
      tc_fence_after();
#pragma unroll
      for (int cb = 0; cb < 4; ++cb) {
        uint32_t pk[16];
        // a block of 32 columns before (behind) all of the warp's rows is full,
        // one behind (before) them empty, the one on the diagonal mixed
        const bool empty = REV ? cb < quad : cb > quad;
        if (empty) {
#pragma unroll
          for (int x = 0; x < 16; ++x) pk[x] = 0u;
        } else {
          float v[32];
          tmem_ld32(tX + lane + cb * 32, v);
          tmem_wait_ld();
          reg_fence<32>(v);
          if (cb != quad && (!REV || nc == kC)) {
            // decay^(i-j) = decay^(distance to the block's near end) times
            // decay^(place within the block): no exponent is negative
            const float f = R.w_in * pw[REV ? cb * 32 - r : r - cb * 32 - 31];
            const float2 ff = make_float2(f, f);
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const float2 u = REV ? make_float2(pw[2 * x], pw[2 * x + 1])
                                   : make_float2(pw[31 - 2 * x], pw[30 - 2 * x]);
              const float2 y = mul2(make_float2(v[2 * x], v[2 * x + 1]), mul2(u, ff));
              pk[x] = pack_bf16x2(y.x, y.y);
            }
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              const int j = cb * 32 + x, gap = REV ? j - r : r - j;
              const bool in = gap >= 0 && (!REV || j < nc);
              v[x] = in ? v[x] * (R.w_in * pw[in ? gap : 0]) : 0.f;
            }
#pragma unroll
            for (int x = 0; x < 16; ++x) pk[x] = pack_bf16x2(v[2 * x], v[2 * x + 1]);
          }
        }
        tmem_st16u(tX + lane + cb * 16, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (tid % 32 == 0) mbar_arrive(b_p);
      if (!(ok = __all_sync(all, wait(b_o, i & 1)))) break;
      tc_fence_after();
      const int row = ch.row(i) + r;
      const int gap = REV ? nc - 1 - r : r;
      const bool real = r < nc;
      const float f = real ? R.w_st * pw[gap + 1 - R.e] : 0.f;
      __nv_bfloat16* dst = out + (i64(bh) * P.N + row) * D;
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        float o[32], z[32];
        tmem_ld32(tO + lane + c, o);
        tmem_ld32(tZ + lane + c, z);
        tmem_wait_ld();
        reg_fence<32>(o);
        reg_fence<32>(z);
        if (c + 32 == D) {
          tc_fence_before();
          __syncwarp();
          if (tid % 32 == 0) mbar_arrive(b_free);
        }
        if (row < P.N) {
#pragma unroll
          for (int x = 0; x < 32; x += 8) {
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (real)
              w = make_uint4(pack_bf16x2(fmaf(f, z[x], o[x]), fmaf(f, z[x + 1], o[x + 1])),
                             pack_bf16x2(fmaf(f, z[x + 2], o[x + 2]), fmaf(f, z[x + 3], o[x + 3])),
                             pack_bf16x2(fmaf(f, z[x + 4], o[x + 4]), fmaf(f, z[x + 5], o[x + 5])),
                             pack_bf16x2(fmaf(f, z[x + 6], o[x + 6]), fmaf(f, z[x + 7], o[x + 7])));
            *reinterpret_cast<uint4*>(dst + c + x) = w;
          }
        }
      }
    }
    // whole chunks behind the sequence's end
    const int seg_end = min(P.seg_len, P.N - ch.t0);
    for (int t = ch.count * kC + r; t < seg_end; t += kC) {
      uint4* dst = reinterpret_cast<uint4*>(out + (i64(bh) * P.N + ch.t0 + t) * D);
#pragma unroll
      for (int x = 0; x < D / 8; ++x) dst[x] = make_uint4(0u, 0u, 0u, 0u);
    }
  } else {
    // ------------------------------------------------ state and weights
    const int r = tid - 128;
    const uint32_t lane = static_cast<uint32_t>(quad * 32) << 16;
    const float* src = starts ? starts + i64(bh) * start_stride + i64(seg) * D * D : nullptr;
    for (int i = 0; ok && i < ch.count; ++i) {
      const int s = i & 1, nc = ch.size(i);
      const float fs = pw[nc];
      if (i > 0) {
        if (!(ok = __all_sync(all, wait(b_s, (i - 1) & 1)))) break;
        tc_fence_after();
      }
      if (r < D) {  // (d = 64: the accumulator's lower rows are not used)
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          float v[32];
          if (i > 0) {
            tmem_ld32(tS + lane + c, v);
            tmem_wait_ld();
            reg_fence<32>(v);
          } else if (!src) {
#pragma unroll
            for (int x = 0; x < 32; ++x) v[x] = 0.f;
          } else if (R.transposed) {
#pragma unroll
            for (int x = 0; x < 32; ++x) v[x] = __ldg(src + (c + x) * D + r);
          } else {
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
              const float4 f4 = __ldg(reinterpret_cast<const float4*>(src + r * D + c + x));
              v[x] = f4.x; v[x + 1] = f4.y; v[x + 2] = f4.z; v[x + 3] = f4.w;
            }
          }
#pragma unroll
          for (int x = 0; x < 32; x += 8) {
            const int u = (c + x) >> 3;
            *reinterpret_cast<uint4*>(base + L::off_s + (u >> 3) * (D * 128) + sw128(r, u & 7)) =
                make_uint4(pack_bf16x2(v[x], v[x + 1]), pack_bf16x2(v[x + 2], v[x + 3]),
                           pack_bf16x2(v[x + 4], v[x + 5]), pack_bf16x2(v[x + 6], v[x + 7]));
          }
#pragma unroll
          for (int x = 0; x < 32; ++x) v[x] *= fs;
          tmem_st32(tS + lane + c, v);
        }
        tmem_wait_st();
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (tid % 32 == 0) mbar_arrive(b_sr);
      // b <- w b in place, X = a b^T having been formed
      if (!(ok = __all_sync(all, wait(b_full + 8 * s, (i >> 1) & 1) && wait(b_x, i & 1)))) break;
      const float w = r < nc ? R.w_sum * pw[(REV ? r : nc - 1 - r) + R.e] : 0.f;
      uint8_t* bt = base + s * L::stage + L::tile;
      constexpr int U = D / 8;
#pragma unroll 8
      for (int u = 0; u < U; ++u) {
        const uint32_t off = (u >> 3) * 16384 + sw128(r, u & 7);
        uint4* p = reinterpret_cast<uint4*>(bt + off);
        uint4 q = *p;
        if (r >= nc) {
          q = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(bt + L::tile + off) = q;  // c: nothing may stand behind a weight of 0
        } else {
          uint32_t* y = reinterpret_cast<uint32_t*>(&q);
#pragma unroll
          for (int x = 0; x < 4; ++x) y[x] = pack_bf16x2(w * lo_bf16(y[x]), w * hi_bf16(y[x]));
        }
        *p = q;
      }
      fence_async_smem();
      __syncwarp();
      if (tid % 32 == 0) mbar_arrive(b_h);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  ok = __syncthreads_and(ok && !*abort_flag);
  drain(ok);
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tX, 512);
  }
}

bool token_map(CUtensorMap* m, const void* ptr, const Geom& g) {
  const uint64_t dims[3] = {static_cast<uint64_t>(g.d), static_cast<uint64_t>(g.N),
                            static_cast<uint64_t>(g.BH)};
  const uint64_t strides[2] = {static_cast<uint64_t>(g.d) * 2, static_cast<uint64_t>(g.N) * g.d * 2};
  const uint32_t box[3] = {64, kC, 1};
  return encode_bf16_map(m, ptr, 3, dims, strides, box);
}

template <typename K>
cudaError_t set_smem(K kern, uint32_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

}  // namespace

int decay_tc_chunk() { return kC; }

bool decay_tc_supported(const Geom& g) {
  return g.dtype == SLA_BF16 && !(g.flags & SLA_FLAG_SIMT);
}

cudaError_t launch_decay_sums_tc(const DecaySums* jobs, int count, const float* log_decay,
                                 const int32_t* lens, const DecayPlan& P, const Geom& g,
                                 int32_t* status, int32_t* zero, cudaStream_t s) {
  CUtensorMap m[4];
  SumsRole r[2];
  for (int i = 0; i < 2; ++i) {
    const DecaySums& j = jobs[i < count ? i : 0];
    if (!token_map(&m[2 * i], j.b, g) || !token_map(&m[2 * i + 1], j.c, g)) return cudaErrorInvalidValue;
    r[i] = SumsRole{j.w_sum, j.e, j.reverse ? 1 : 0};
  }
  const dim3 grid(P.segs, g.BH, count);
  const int hold = debug_withhold(g, SLA_WITHHOLD_SUMMARIES) ? 1 : 0;
  float* s1 = jobs[count - 1].sums;
  auto go = [&](auto kern, uint32_t smem) {
    cudaError_t e = set_smem(kern, smem);
    if (e != cudaSuccess) return e;
    kern<<<grid, kThreads, smem, s>>>(m[0], m[1], m[2], m[3], log_decay, lens, jobs[0].sums, s1, P, r[0],
                                      r[1], status, zero, wait_limit(g), hold);
    return cudaGetLastError();
  };
  return g.d == 128 ? go(decay_sums_tc<128>, SumsSmem<128>::total) : go(decay_sums_tc<64>, SumsSmem<64>::total);
}

cudaError_t launch_decay_out_tc(const void* a, const void* b, const void* c, const float* log_decay,
                                const int32_t* lens, const float* starts, i64 start_stride, void* out,
                                const DecayPlan& P, const DecayRole& R, const Geom& g, int32_t* status,
                                int32_t* zero, cudaStream_t s) {
  CUtensorMap ma, mb, mc;
  if (!token_map(&ma, a, g) || !token_map(&mb, b, g) || !token_map(&mc, c, g)) return cudaErrorInvalidValue;
  const int hold = debug_withhold(g, SLA_WITHHOLD_ATTENTION) ? 1 : 0;
  auto go = [&](auto kern, uint32_t smem) {
    cudaError_t e = set_smem(kern, smem);
    if (e != cudaSuccess) return e;
    kern<<<dim3(P.segs, g.BH), kThreads, smem, s>>>(ma, mb, mc, log_decay, lens, starts, start_stride,
                                                    static_cast<__nv_bfloat16*>(out), P, R, status, zero,
                                                    wait_limit(g), hold);
    return cudaGetLastError();
  };
  if (g.d == 128)
    return R.reverse ? go(decay_out_tc<128, true>, OutSmem<128>::total)
                     : go(decay_out_tc<128, false>, OutSmem<128>::total);
  return R.reverse ? go(decay_out_tc<64, true>, OutSmem<64>::total)
                   : go(decay_out_tc<64, false>, OutSmem<64>::total);
}

}  // namespace sla
