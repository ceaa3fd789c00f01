// Linear attention with a decay for each head: fp32 kernels, the scan over
// segments, and the single-token form.
//
// With g = log_decay[h] and state S (d x d, row = channel of b, column =
// channel of c), one operation covers the forward and all three gradients:
//   out_i = w_in sum_{j <= i} e^{g (i-j)} (a_i . b_j) c_j + w_st e^{g (i+1-e)} a_i S
//   S'    = e^{g n} S + w_sum sum_j e^{g (n-1-j+e)} b_j^T c_j
// over the n tokens of a piece counted from the side where S enters:
//   forward     a, b, c = q, k, v         first to last   e = 0
//   dq          a, b, c = dout, v, k      first to last   e = 0   state S^T
//   dv          a, b, c = k, q, dout      last to first   e = 1   state R
//   dk          a, b, c = v, dout, q      last to first   e = 1   state R^T
// where R is the gradient of the state (e: the output is formed from the
// state that holds its own token, so the gradient reaches one step further).
//
// A sequence is cut into segments that run in parallel: (1) each segment's
// own sum, (2) a scan that turns the sums into the states at the segments'
// starts, (3) the outputs, each segment walked chunk by chunk with its state
// on chip.  One segment needs (3) only.
#include <algorithm>

#include "common.cuh"
#include "decay.cuh"

namespace sla {

namespace {

constexpr int kC = 32;        // tokens per chunk of the fp32 kernels
constexpr int kThr = 256;

// The workspace's status word, cleared by the first kernel of a call.
__device__ __forceinline__ void zero_word(int32_t* w) {
  if (w && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *w = 0;
}

// Rows [r0, r0 + kC) (by counted index i within the piece of n tokens at t0)
// of one head's [N, d] tensor into smem as fp32; rows at or past n are zero.
template <typename T, int D>
__device__ __forceinline__ void load_rows(const T* __restrict__ x, float* dst, int i0, int n, int t0,
                                          bool reverse) {
  for (int u = threadIdx.x; u < kC * (D / 4); u += kThr) {
    const int r = u / (D / 4), c = (u % (D / 4)) * 4;
    const int i = i0 + r;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < n) f = load4(x + i64(t0 + (reverse ? n - 1 - i : i)) * D + c);
    *reinterpret_cast<float4*>(dst + r * (D + 4) + c) = f;
  }
}

// S (smem, [D][D + 4]) <- f S + sum over the chunk's rows of w_r b_r^T c_r;
// each thread owns D * D / 256 elements: rows ty + 16 x, columns 4 tx + 64 y
template <int D>
__device__ __forceinline__ void add_outer(float* S, const float* b, const float* c, const float* w,
                                          float2 f) {
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  constexpr int LD = D + 4, RX = D / 16, CY = D / 64;
  float acc[RX][CY * 4];
#pragma unroll
  for (int x = 0; x < RX; ++x)
#pragma unroll
    for (int y = 0; y < CY; ++y) {
      const float4 s = *reinterpret_cast<const float4*>(S + (ty + 16 * x) * LD + 4 * tx + 64 * y);
      acc[x][4 * y] = times(f, s.x); acc[x][4 * y + 1] = times(f, s.y);
      acc[x][4 * y + 2] = times(f, s.z); acc[x][4 * y + 3] = times(f, s.w);
    }
#pragma unroll 4
  for (int r = 0; r < kC; ++r) {
    float cv[CY * 4];
    const float wr = w[r];
#pragma unroll
    for (int y = 0; y < CY; ++y) {
      const float4 v = *reinterpret_cast<const float4*>(c + r * LD + 4 * tx + 64 * y);
      cv[4 * y] = wr * v.x; cv[4 * y + 1] = wr * v.y; cv[4 * y + 2] = wr * v.z; cv[4 * y + 3] = wr * v.w;
    }
#pragma unroll
    for (int x = 0; x < RX; ++x) {
      const float bv = b[r * LD + ty + 16 * x];
#pragma unroll
      for (int y = 0; y < CY * 4; ++y) acc[x][y] = fmaf(bv, cv[y], acc[x][y]);
    }
  }
#pragma unroll
  for (int x = 0; x < RX; ++x)
#pragma unroll
    for (int y = 0; y < CY; ++y)
      *reinterpret_cast<float4*>(S + (ty + 16 * x) * LD + 4 * tx + 64 * y) =
          make_float4(acc[x][4 * y], acc[x][4 * y + 1], acc[x][4 * y + 2], acc[x][4 * y + 3]);
}

// S from global [D][D], transposed if asked
template <int D>
__device__ __forceinline__ void load_state(float* S, const float* src, bool transposed) {
#pragma unroll 4
  for (int u = threadIdx.x; u < D * D / 4; u += kThr) {
    const int r = u / (D / 4), c = u % (D / 4) * 4;
    const float4 f = src ? *reinterpret_cast<const float4*>(src + 4 * u) : make_float4(0.f, 0.f, 0.f, 0.f);
    if (transposed) {
      S[c * (D + 4) + r] = f.x;
      S[(c + 1) * (D + 4) + r] = f.y;
      S[(c + 2) * (D + 4) + r] = f.z;
      S[(c + 3) * (D + 4) + r] = f.w;
    } else {
      *reinterpret_cast<float4*>(S + r * (D + 4) + c) = f;
    }
  }
}

// (1) sums of the segments: sums[bh][seg] = w_sum sum_i e^{g (n-1-i+e)} b_i^T c_i
template <typename T, int D>
__global__ void __launch_bounds__(kThr) decay_sums_simt(const T* __restrict__ b, const T* __restrict__ c,
                                                        const float* __restrict__ log_decay,
                                                        const int32_t* __restrict__ lens,
                                                        float* __restrict__ sums, DecayPlan P, int e,
                                                        bool reverse, float w_sum, int32_t* zero) {
  next_may_launch();
  zero_word(zero);
  extern __shared__ float sm[];
  float* S = sm;
  float* bt = S + D * (D + 4);
  float* ct = bt + kC * (D + 4);
  __shared__ float w[kC];
  const int bh = blockIdx.y, seg = blockIdx.x;
  const double l2 = decay_log2(log_decay[bh % P.H]);
  const int t0 = seg * P.seg_len, n = segment_tokens(P, lens, bh / P.H, seg);
  const i64 base = i64(bh) * P.N * D;
  load_state<D>(S, nullptr, false);
  for (int i0 = 0; i0 < n; i0 += kC) {
    __syncthreads();
    load_rows<T, D>(b + base, bt, i0, n, t0, reverse);
    load_rows<T, D>(c + base, ct, i0, n, t0, reverse);
    // weights count from the segment's end: nothing is scaled again later
    if (threadIdx.x < kC) {
      const int left = n - 1 - i0 - static_cast<int>(threadIdx.x);
      w[threadIdx.x] = left >= 0 ? w_sum * decay_power(l2, left + e) : 0.f;
    }
    __syncthreads();
    add_outer<D>(S, bt, ct, w, make_float2(1.f, 0.f));
  }
  __syncthreads();
  float* dst = sums + (i64(bh) * P.segs + seg) * D * D;
  for (int u = threadIdx.x; u < D * D; u += kThr) dst[u] = S[u / D * (D + 4) + u % D];
}

// (3) outputs of a segment
template <typename T, int D>
__global__ void __launch_bounds__(kThr) decay_out_simt(const T* __restrict__ a, const T* __restrict__ b,
                                                       const T* __restrict__ c,
                                                       const float* __restrict__ log_decay,
                                                       const int32_t* __restrict__ lens,
                                                       const float* starts, i64 start_stride,
                                                       T* __restrict__ out, float* final_state,
                                                       DecayPlan P, DecayRole R, int32_t* zero) {
  next_may_launch();
  zero_word(zero);
  extern __shared__ float sm[];
  constexpr int LD = D + 4;
  float* S = sm;
  float* at = S + D * LD;
  float* bt = at + kC * LD;
  float* ct = bt + kC * LD;
  float* pt = ct + kC * LD;  // [kC][kC + 1]
  __shared__ float w[kC], pw[kC + 1];
  const int bh = blockIdx.y, seg = blockIdx.x;
  const double l2 = decay_log2(log_decay[bh % P.H]);
  const int t0 = seg * P.seg_len, n = segment_tokens(P, lens, bh / P.H, seg);
  const i64 base = i64(bh) * P.N * D;
  if (threadIdx.x <= kC) pw[threadIdx.x] = decay_power(l2, threadIdx.x);
  const bool moves = n > kC || final_state;  // whether the state is taken on at all
  const float2 full = moves ? decay_power2(l2, kC) : make_float2(0.f, 0.f);
  wait_for_previous();
  load_state<D>(S, starts ? starts + i64(bh) * start_stride + i64(seg) * D * D : nullptr, R.transposed);
  for (int i0 = 0; i0 < n; i0 += kC) {
    __syncthreads();
    load_rows<T, D>(a + base, at, i0, n, t0, R.reverse);
    load_rows<T, D>(b + base, bt, i0, n, t0, R.reverse);
    load_rows<T, D>(c + base, ct, i0, n, t0, R.reverse);
    const int nc = min(kC, n - i0);
    if (threadIdx.x < kC)
      w[threadIdx.x] = threadIdx.x < nc ? R.w_sum * decay_power(l2, nc - 1 - threadIdx.x + R.e) : 0.f;
    __syncthreads();
    // scores: 4 per thread
    {
      const int j = threadIdx.x % 32, r = threadIdx.x / 32;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int k = 0; k < D; k += 4) {
        const float4 y = *reinterpret_cast<const float4*>(bt + j * LD + k);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float4 q = *reinterpret_cast<const float4*>(at + (r + 8 * x) * LD + k);
          acc[x] += q.x * y.x + q.y * y.y + q.z * y.z + q.w * y.w;
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int i = r + 8 * x;
        pt[i * (kC + 1) + j] = j <= i ? R.w_in * pw[i - j] * acc[x] : 0.f;
      }
    }
    __syncthreads();
    // outputs: rows r + 8 x, 4 columns per lane and 128-wide pass
    {
      constexpr int LANES = D / 4;           // lanes that cover a row
      constexpr int RPP = kThr / LANES;      // rows per pass
      const int col = threadIdx.x % LANES * 4, r = threadIdx.x / LANES;
      constexpr int X = kC / RPP;
      float4 y[X], z[X];
#pragma unroll
      for (int x = 0; x < X; ++x) y[x] = z[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int j = 0; j < kC; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(ct + j * LD + col);
#pragma unroll
        for (int x = 0; x < X; ++x) {
          const float p = pt[(r + RPP * x) * (kC + 1) + j];
          y[x].x = fmaf(p, v.x, y[x].x); y[x].y = fmaf(p, v.y, y[x].y);
          y[x].z = fmaf(p, v.z, y[x].z); y[x].w = fmaf(p, v.w, y[x].w);
        }
      }
#pragma unroll 4
      for (int k = 0; k < D; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(S + k * LD + col);
#pragma unroll
        for (int x = 0; x < X; ++x) {
          const float q = at[(r + RPP * x) * LD + k];
          z[x].x = fmaf(q, v.x, z[x].x); z[x].y = fmaf(q, v.y, z[x].y);
          z[x].z = fmaf(q, v.z, z[x].z); z[x].w = fmaf(q, v.w, z[x].w);
        }
      }
#pragma unroll
      for (int x = 0; x < X; ++x) {
        const int i = i0 + r + RPP * x;
        if (i < n) {
          const float f = R.w_st * pw[r + RPP * x + 1 - R.e];
          store4(out + base + i64(t0 + (R.reverse ? n - 1 - i : i)) * D + col,
                 make_float4(y[x].x + f * z[x].x, y[x].y + f * z[x].y, y[x].z + f * z[x].z,
                             y[x].w + f * z[x].w));
        }
      }
    }
    if (i0 + kC >= n && !final_state) break;  // nobody reads the state behind this chunk
    __syncthreads();
    add_outer<D>(S, bt, ct, w, nc == kC ? full : decay_power2(l2, nc));
  }
  // rows behind the sequence's end
  const int pad = min(P.seg_len, P.N - t0) - n;
  for (int u = threadIdx.x; u < pad * (D / 4); u += kThr)
    store4(out + base + i64(t0 + n) * D + u * 4, make_float4(0.f, 0.f, 0.f, 0.f));
  if (final_state) {
    __syncthreads();
    float* dst = final_state + i64(bh) * D * D;
    for (int u = threadIdx.x; u < D * D; u += kThr) {
      const int r = u / D, c2 = u % D;
      dst[u] = S[(R.transposed ? c2 : r) * LD + (R.transposed ? r : c2)];
    }
  }
}

// (2) The sums of a head's segments -> the state at each one's entering side,
// in place; the state behind the last one -> final_state.  One thread per 4
// elements, segments in the walk's order: sums are read and written once (they
// sit in L2), the order of the additions is fixed.
//
// The segments are the uniform ones of the fp32 kernels, or the pieces of the
// tensor-core kernels with their packed sums (units of 4 columns, rows
// adjacent).  Each block first tables its head's segments: place and factor.
struct UniformSegments {
  DecayPlan P;
  static constexpr bool packed = false;
  __device__ int first(int) const { return 0; }
  __device__ int count(int) const { return P.segs; }
  __device__ int begin(int, int i) const { return i * P.seg_len; }
  __device__ int place(int bh, int i) const { return bh * P.segs + i; }
};
struct PieceSegments {
  DecayParts P;
  static constexpr bool packed = true;
  __device__ int first(int bh) const { return P.part(i64(bh) * P.chunks); }
  __device__ int count(int bh) const { return P.part(i64(bh + 1) * P.chunks - 1) - first(bh) + 1; }
  // first token of part k within head bh
  __device__ int begin(int bh, int k) const {
    return static_cast<int>(min(max(P.begin(k) - i64(bh) * P.chunks, i64(0)), i64(P.chunks))) * 128;
  }
  __device__ int place(int bh, int k) const { return k + bh; }
};

constexpr int kScan = 14;      // segments' sums in flight per thread
constexpr int kScanTable = 512;  // segments of a head tabled at a time
template <typename Segments>
__global__ void __launch_bounds__(128) decay_scan_kernel(DecayScanJob j0, DecayScanJob j1,
                                                         const float* __restrict__ log_decay,
                                                         const int32_t* __restrict__ lens, Segments G,
                                                         int d) {
  next_may_launch();
  __shared__ float2 factor[kScanTable];
  __shared__ int place[kScanTable];
  const DecayScanJob J = blockIdx.z ? j1 : j0;
  float4* sums = reinterpret_cast<float4*>(J.sums);
  const int dd4 = d * d / 4;
  const int u = blockIdx.x * 128 + threadIdx.x;
  const int bh = blockIdx.y;
  const int r = G.packed ? u % d : u / (d / 4), c = G.packed ? u / d * 4 : u % (d / 4) * 4;
  const double l2 = decay_log2(log_decay[bh % G.P.H]);
  const int len = decay_tokens(lens, bh / G.P.H, G.P.N);
  const int segs = G.count(bh), seg0 = G.first(bh);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (J.first) {
    const float* f = J.first + i64(bh) * d * d;
    s = J.turned ? make_float4(f[c * d + r], f[(c + 1) * d + r], f[(c + 2) * d + r], f[(c + 3) * d + r])
                 : *reinterpret_cast<const float4*>(f + r * d + c);
  }
  for (int t0 = 0; t0 < segs; t0 += kScanTable) {
    const int tn = min(kScanTable, segs - t0);
    __syncthreads();
    for (int i = threadIdx.x; i < tn; i += 128) {
      const int k = seg0 + (J.reverse ? segs - 1 - (t0 + i) : t0 + i);
      const int b0 = G.begin(bh, k), b1 = G.begin(bh, k + 1);
      factor[i] = decay_power2(l2, min(max(len - b0, 0), b1 - b0));
      place[i] = G.place(bh, k);
    }
    __syncthreads();
    if (t0 == 0) wait_for_previous();
    for (int i0 = 0; i0 < tn; i0 += kScan) {
      float4 x[kScan];
#pragma unroll
      for (int i = 0; i < kScan; ++i)
        if (i0 + i < tn) x[i] = sums[i64(place[i0 + i]) * dd4 + u];
#pragma unroll
      for (int i = 0; i < kScan; ++i) {
        if (i0 + i < tn) {
          sums[i64(place[i0 + i]) * dd4 + u] = s;
          const float2 f = factor[i0 + i];
          s.x = fmaf(f.x, s.x, fmaf(f.y, s.x, x[i].x)); s.y = fmaf(f.x, s.y, fmaf(f.y, s.y, x[i].y));
          s.z = fmaf(f.x, s.z, fmaf(f.y, s.z, x[i].z)); s.w = fmaf(f.x, s.w, fmaf(f.y, s.w, x[i].w));
        }
      }
    }
  }
  if (J.last) reinterpret_cast<float4*>(J.last)[i64(bh) * dd4 + r * (d / 4) + c / 4] = s;
}

// Few tokens: the state is read and written once, by CTAs that own 32 columns
// of one head's state each (128-byte rows; 8 threads x 4 columns, 32 groups
// of D / 32 rows), tokens one after another with the state in registers.
// Bound by the states' traffic, 8 d^2 bytes per head.
template <typename T, int D>
__global__ void __launch_bounds__(256) decay_step_kernel(const T* __restrict__ q, const T* __restrict__ k,
                                                         const T* __restrict__ v,
                                                         const float* __restrict__ log_decay,
                                                         const int32_t* __restrict__ lens,
                                                         const float* state_in, float* state_out,
                                                         T* __restrict__ out, int N, int H, float scale,
                                                         int32_t* zero) {
  zero_word(zero);
  constexpr int R = D / 32;
  __shared__ float red[8][32];
  const int bh = blockIdx.x, col0 = blockIdx.y * 32;
  const int cx = threadIdx.x % 8 * 4, rg = threadIdx.x / 8, warp = threadIdx.x / 32;
  const float f = decay_power(decay_log2(log_decay[bh % H]), 1);
  const int n = lens ? min(max(lens[bh / H], 0), N) : N;
  const i64 sbase = i64(bh) * D * D + col0 + cx;
  float4 s[R];
#pragma unroll
  for (int x = 0; x < R; ++x)
    s[x] = state_in ? *reinterpret_cast<const float4*>(state_in + sbase + i64(rg * R + x) * D)
                    : make_float4(0.f, 0.f, 0.f, 0.f);
  const i64 base = i64(bh) * N * D;
  for (int t = 0; t < N; ++t) {
    if (t >= n) {  // uniform over the CTA
      if (threadIdx.x < 32) out[base + t * D + col0 + threadIdx.x] = from_f32<T>(0.f);
      continue;
    }
    const float4 vv = load4(v + base + t * D + col0 + cx);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int x = 0; x < R; ++x) {
      const float kk = to_f32(k[base + t * D + rg * R + x]), qq = to_f32(q[base + t * D + rg * R + x]);
      s[x].x = fmaf(f, s[x].x, kk * vv.x); s[x].y = fmaf(f, s[x].y, kk * vv.y);
      s[x].z = fmaf(f, s[x].z, kk * vv.z); s[x].w = fmaf(f, s[x].w, kk * vv.w);
      o.x = fmaf(qq, s[x].x, o.x); o.y = fmaf(qq, s[x].y, o.y);
      o.z = fmaf(qq, s[x].z, o.z); o.w = fmaf(qq, s[x].w, o.w);
    }
#pragma unroll
    for (int m = 8; m < 32; m *= 2) {
      o.x += __shfl_xor_sync(0xffffffffu, o.x, m);
      o.y += __shfl_xor_sync(0xffffffffu, o.y, m);
      o.z += __shfl_xor_sync(0xffffffffu, o.z, m);
      o.w += __shfl_xor_sync(0xffffffffu, o.w, m);
    }
    if (threadIdx.x % 32 < 8) *reinterpret_cast<float4*>(&red[warp][cx]) = o;
    __syncthreads();
    if (threadIdx.x < 32) {
      float y = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) y += red[w][threadIdx.x];
      out[base + t * D + col0 + threadIdx.x] = from_f32<T>(scale * y);
    }
    __syncthreads();
  }
  if (state_out && (n > 0 || state_out != state_in)) {
#pragma unroll
    for (int x = 0; x < R; ++x)
      *reinterpret_cast<float4*>(state_out + sbase + i64(rg * R + x) * D) = s[x];
  }
}

template <typename T, int D>
cudaError_t sums_simt(const T* b, const T* c, const float* ld, const int32_t* lens, float* sums,
                      const DecayPlan& P, int e, bool reverse, float w_sum, int BH, int32_t* zero,
                      cudaStream_t s) {
  const size_t smem = sizeof(float) * (D + 2 * kC) * (D + 4);
  auto kern = decay_sums_simt<T, D>;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (err != cudaSuccess) return err;
  kern<<<dim3(P.segs, BH), kThr, smem, s>>>(b, c, ld, lens, sums, P, e, reverse, w_sum, zero);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t out_simt(const T* a, const T* b, const T* c, const float* ld, const int32_t* lens,
                     const float* starts, i64 stride, T* out, float* fin, const DecayPlan& P,
                     const DecayRole& R, int BH, int32_t* zero, cudaStream_t s) {
  const size_t smem = sizeof(float) * ((D + 3 * kC) * (D + 4) + kC * (kC + 1));
  auto kern = decay_out_simt<T, D>;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (err != cudaSuccess) return err;
  // (the first kernel of a call clears the status word)
  return launch_behind(!zero, kern, dim3(P.segs, BH), kThr, smem, s, a, b, c, ld, lens, starts, stride, out,
                       fin, P, R, zero);
}

}  // namespace

int decay_simt_chunk() { return kC; }

cudaError_t launch_decay_sums_simt(const void* b, const void* c, const float* log_decay,
                                   const int32_t* lens, float* sums, const DecayPlan& P, int e,
                                   bool reverse, float w_sum, const Geom& g, int32_t* zero,
                                   cudaStream_t s) {
  using bf = __nv_bfloat16;
  if (g.dtype == SLA_F32) {
    const float *x = static_cast<const float*>(b), *y = static_cast<const float*>(c);
    return g.d == 64 ? sums_simt<float, 64>(x, y, log_decay, lens, sums, P, e, reverse, w_sum, g.BH, zero, s)
                     : sums_simt<float, 128>(x, y, log_decay, lens, sums, P, e, reverse, w_sum, g.BH, zero, s);
  }
  const bf *x = static_cast<const bf*>(b), *y = static_cast<const bf*>(c);
  return g.d == 64 ? sums_simt<bf, 64>(x, y, log_decay, lens, sums, P, e, reverse, w_sum, g.BH, zero, s)
                   : sums_simt<bf, 128>(x, y, log_decay, lens, sums, P, e, reverse, w_sum, g.BH, zero, s);
}

cudaError_t launch_decay_out_simt(const void* a, const void* b, const void* c, const float* log_decay,
                                  const int32_t* lens, const float* starts, i64 start_stride, void* out,
                                  float* final_state, const DecayPlan& P, const DecayRole& R,
                                  const Geom& g, int32_t* zero, cudaStream_t s) {
  using bf = __nv_bfloat16;
  if (g.dtype == SLA_F32) {
    const float *x = static_cast<const float*>(a), *y = static_cast<const float*>(b),
                *z = static_cast<const float*>(c);
    float* o = static_cast<float*>(out);
    return g.d == 64 ? out_simt<float, 64>(x, y, z, log_decay, lens, starts, start_stride, o, final_state, P, R, g.BH, zero, s)
                     : out_simt<float, 128>(x, y, z, log_decay, lens, starts, start_stride, o, final_state, P, R, g.BH, zero, s);
  }
  const bf *x = static_cast<const bf*>(a), *y = static_cast<const bf*>(b), *z = static_cast<const bf*>(c);
  bf* o = static_cast<bf*>(out);
  return g.d == 64 ? out_simt<bf, 64>(x, y, z, log_decay, lens, starts, start_stride, o, final_state, P, R, g.BH, zero, s)
                   : out_simt<bf, 128>(x, y, z, log_decay, lens, starts, start_stride, o, final_state, P, R, g.BH, zero, s);
}

cudaError_t launch_decay_scan(const DecayScanJob& job, const float* log_decay, const int32_t* lens,
                              const DecayPlan& P, const Geom& g, cudaStream_t s) {
  return launch_behind(true, decay_scan_kernel<UniformSegments>, dim3(g.d * g.d / 512, g.BH), 128, 0, s,
                       job, job, log_decay, lens, UniformSegments{P}, g.d);
}

cudaError_t launch_decay_scan_parts(const DecayScanJob* jobs, int count, const float* log_decay,
                                    const int32_t* lens, const DecayParts& P, const Geom& g,
                                    cudaStream_t s) {
  return launch_behind(true, decay_scan_kernel<PieceSegments>, dim3(g.d * g.d / 512, g.BH, count), 128, 0,
                       s, jobs[0], jobs[count - 1], log_decay, lens, PieceSegments{P}, g.d);
}

cudaError_t launch_decay_step(const void* q, const void* k, const void* v, const float* log_decay,
                              const int32_t* lens, const float* state_in, float* state_out, void* out,
                              const Geom& g, int32_t* zero, cudaStream_t s) {
  using bf = __nv_bfloat16;
  const dim3 grid(g.BH, g.d / 32);
  auto run = [&](auto kern, auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    kern<<<grid, 256, 0, s>>>(static_cast<const T*>(q), static_cast<const T*>(k),
                              static_cast<const T*>(v), log_decay, lens, state_in, state_out,
                              static_cast<T*>(out), g.N, g.H, g.scale, zero);
    return cudaGetLastError();
  };
  if (g.dtype == SLA_F32)
    return g.d == 64 ? run(decay_step_kernel<float, 64>, static_cast<float*>(nullptr))
                     : run(decay_step_kernel<float, 128>, static_cast<float*>(nullptr));
  return g.d == 64 ? run(decay_step_kernel<bf, 64>, static_cast<bf*>(nullptr))
                   : run(decay_step_kernel<bf, 128>, static_cast<bf*>(nullptr));
}

}  // namespace sla
