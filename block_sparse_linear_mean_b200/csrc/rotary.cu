// Rotary positions: q and k turned by their tokens' positions, and their
// gradients back.
//
// Pair (a, b) of a token at position x turns by the angle x w:
//   a' = m (a cos - b sin),  b' = m (b cos + a sin);   the transpose (the
// gradient) has -sin.  The pass reads the projection's layout (any strides),
// takes tokens into another order on the way and writes the dense [B,H,N,d]
// that mask and attention read, or goes the other way.
//
// Angles: x w is formed in 64 bits and reduced to a fraction of a turn there,
// so a position of a million still has its phase to 2^-25 of a turn (in 32
// bits the product alone would be off by 0.03 rad); sine and cosine of the
// fraction are fp32.  They are shared by all heads, so a thread keeps the
// cosines of its few pairs of one token in registers and walks over the heads
// of both tensors: one 64-bit angle per (token, pair), not per value.
//
// Bound by HBM: every value is read once and written once.  q and k of 12 heads
// of 32,760 tokens, d = 128, bf16, from the projection's layout into tile order
// and the dense one: 403 MB in 66 us (6.1 TB/s); gradients in fp32 back, 604 MB
// in 92 us (6.6 TB/s).  Rows wait in the words they are stored in, not as fp32,
// so that four CTAs fit an SM (62 registers): 99 us before that, 76 with three.
#include <algorithm>

#include "common.cuh"

namespace sla {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 64;
constexpr int kWords = 32;  // 4-byte words in flight per thread

// The side that is read and the side that is written, in elements.
struct Side {
  i64 b, h, n;
};

struct RotaryArgs {
  const void* src[2];
  void* dst[2];
  Side in, out;
  const int32_t* positions;  // [axes, N] or [B, axes, N]
  const int32_t* perm;
  i64 tokens;                // B * N
  int N, H, d;
  int tensors;               // 1 or 2
  int rows_per_group;        // rows = (tensor, head) pairs per blockIdx.y
  int pairs, axes;
  int split1, split2;        // first pair of axes 1 and 2
  int grid_r, grid_c;
  int origin[3];
  int pos_batched;
  int gather;                // perm on the read side (forward) or the written one
  float sign, amplitude;
  double turns[kMaxPairs];   // freq / 2 pi
};

// V consecutive elements of a row, as the words they are stored in: rows in
// flight cost registers by their bytes, not as fp32.
template <typename T, int V>
struct Words {
  static constexpr int bytes = V * static_cast<int>(sizeof(T));
  static constexpr int n = bytes < 4 ? 1 : bytes / 4;
  uint32_t w[n];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (bytes >= 16) {
#pragma unroll
      for (int i = 0; i < n; i += 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) + 4 * i);
        w[i] = u.x; w[i + 1] = u.y; w[i + 2] = u.z; w[i + 3] = u.w;
      }
    } else if constexpr (bytes == 8) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x; w[1] = u.y;
    } else if constexpr (bytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (bytes >= 16) {
#pragma unroll
      for (int i = 0; i < n; i += 4)
        *reinterpret_cast<uint4*>(reinterpret_cast<char*>(p) + 4 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else if constexpr (bytes == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else if constexpr (bytes == 4) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
      *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
  // elements i and i + 1 (i even), or the only one
  __device__ __forceinline__ void put(int i, float a, float b) {
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(a);
      if constexpr (V > 1) w[i + 1] = __float_as_uint(b);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      w[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
};

// A unit is V pairs of one token's row (2 V channels); the d / (2 V) units of
// a row take one thread each.  The first `pairs` pairs turn, the rest are copied.
// Half layout: channels [a, a + V) and [a + pairs, + V), and V divides `pairs`;
// interleaved: 2 V neighbours, and a unit may turn some of its pairs only.
template <typename TIn, typename TOut, int V, bool INTER>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const __grid_constant__ RotaryArgs A) {
  __shared__ double turns[kMaxPairs];
  if (threadIdx.x < kMaxPairs) turns[threadIdx.x] = A.turns[threadIdx.x];
  __syncthreads();
  const int units = A.d / (2 * V);
  const int per_cta = kThreads / units;
  const int u = threadIdx.x % units;
  const i64 tok = i64(blockIdx.x) * per_cta + threadIdx.x / units;
  if (tok >= A.tokens) return;
  const i64 b = tok / A.N;
  const int n = static_cast<int>(tok - b * A.N);
  int t = n;  // raw token
  if (A.perm) {
    t = A.perm[n];
    if (t < 0 || t >= A.N) return;
  }
  const int turned = A.pairs - u * V;  // pairs of the unit that turn, if positive
  const bool turn = turned > 0;
  float cs[V], sn[V];
  if (turn) {
    i64 pos[3];
    if (A.positions) {
      const int32_t* ps = A.positions + (A.pos_batched ? b * A.axes : 0) * A.N + t;
      pos[0] = ps[0];
      pos[1] = A.axes > 1 ? ps[A.N] : 0;
      pos[2] = A.axes > 2 ? ps[i64(A.N) * 2] : 0;
    } else if (A.axes == 1) {
      pos[0] = i64(t) + A.origin[0];
      pos[1] = pos[2] = 0;
    } else {
      const int c = t % A.grid_c, fr = t / A.grid_c;
      if (A.axes == 2) {
        pos[0] = i64(fr) + A.origin[0];
        pos[1] = i64(c) + A.origin[1];
        pos[2] = 0;
      } else {
        pos[0] = i64(fr / A.grid_r) + A.origin[0];
        pos[1] = i64(fr % A.grid_r) + A.origin[1];
        pos[2] = i64(c) + A.origin[2];
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = u * V + i;
      const i64 x = c < A.split1 ? pos[0] : c < A.split2 ? pos[1] : pos[2];
      const double ang = static_cast<double>(x) * turns[c];
      float s, co;
      sincospif(2.f * static_cast<float>(ang - rint(ang)), &s, &co);
      cs[i] = co * A.amplitude;
      sn[i] = s * A.amplitude * A.sign;
    }
  }
  // first channels of the unit's two pieces of V
  int c0, c1;
  if (INTER) {
    c0 = 2 * V * u;
    c1 = c0 + V;
  } else if (turn) {
    c0 = u * V;
    c1 = c0 + A.pairs;
  } else {
    c0 = 2 * A.pairs + 2 * (u * V - A.pairs);
    c1 = c0 + V;
  }
  const int n_in = A.gather ? t : n, n_out = A.gather ? n : t;
  const i64 in0 = b * A.in.b + n_in * A.in.n, out0 = b * A.out.b + n_out * A.out.n;
  const int row0 = blockIdx.y * A.rows_per_group;
  const int row1 = min(row0 + A.rows_per_group, A.tensors * A.H);
  // INTER: one access of 2 V; half: one of V for each piece
  constexpr int VA = INTER ? 2 * V : V;
  using In = Words<TIn, VA>;
  using Out = Words<TOut, VA>;
  constexpr int per_row = In::n * (INTER ? 1 : 2);
  constexpr int kRows = kWords / per_row < 8 ? kWords / per_row : 8;
  for (int r0 = row0; r0 < row1; r0 += kRows) {
    In x[kRows][INTER ? 1 : 2];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int r = r0 + k;
      if (r < row1) {
        const int second = r >= A.H, h = second ? r - A.H : r;
        const TIn* src = static_cast<const TIn*>(second ? A.src[1] : A.src[0]) + in0 + h * A.in.h;
        x[k][0].load(src + c0);
        if constexpr (!INTER) x[k][1].load(src + c1);
      }
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int r = r0 + k;
      if (r < row1) {
        const int second = r >= A.H, h = second ? r - A.H : r;
        TOut* dst = static_cast<TOut*>(second ? A.dst[1] : A.dst[0]) + out0 + h * A.out.h;
        if constexpr (INTER) {
          Out y;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float a = x[k][0].get(2 * i), b = x[k][0].get(2 * i + 1);
            y.put(2 * i, i < turned ? a * cs[i] - b * sn[i] : a, i < turned ? b * cs[i] + a * sn[i] : b);
          }
          y.store(dst + c0);
        } else {
          Out y, z;
#pragma unroll
          for (int i = 0; i < V; i += 2) {
            const int j = V > 1 ? i + 1 : i;
            const float a0 = x[k][0].get(i), b0 = x[k][1].get(i), a1 = x[k][0].get(j), b1 = x[k][1].get(j);
            y.put(i, turn ? a0 * cs[i] - b0 * sn[i] : a0, turn ? a1 * cs[j] - b1 * sn[j] : a1);
            z.put(i, turn ? b0 * cs[i] + a0 * sn[i] : b0, turn ? b1 * cs[j] + a1 * sn[j] : b1);
          }
          y.store(dst + c0);
          z.store(dst + c1);
        }
      }
    }
  }
}

template <typename TIn, typename TOut, int V, bool INTER>
cudaError_t launch(RotaryArgs& a, cudaStream_t s) {
  const int per_cta = kThreads / (a.d / (2 * V));
  const i64 gx = (a.tokens + per_cta - 1) / per_cta;
  const int rows = a.tensors * a.H;
  // few tokens: the rows are spread over more CTAs (their angles are formed
  // again there), down to two rows each (one token of 12 heads: 3.2 us, in one
  // CTA 13.5)
  const i64 want = std::max<i64>(1, 148 * 4 / gx);
  const int groups = static_cast<int>(std::min<i64>(want, std::max(1, rows / 2)));
  a.rows_per_group = (rows + groups - 1) / groups;
  const dim3 grid(static_cast<unsigned>(gx), (rows + a.rows_per_group - 1) / a.rows_per_group);
  rotary_kernel<TIn, TOut, V, INTER><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename TIn, typename TOut>
cudaError_t dispatch(RotaryArgs& a, bool inter, cudaStream_t s) {
  // Pairs per unit: four (interleaved bf16 moves 16 bytes per access, half
  // layout twice 8), two in interleaved fp32 (16 bytes); in half layout fewer
  // where the split at `pairs` asks for it.  q and k of 12 heads of 32,760
  // tokens, d = 128, bf16: 66 us in both layouts; with two pairs 79
  // (interleaved) and 85 us (half), with one 138 and 135; with eight, half, 81:
  // fewer rows in flight.
  const int p = a.pairs;
  if (inter) return launch<TIn, TOut, sizeof(TIn) == 2 || sizeof(TOut) == 2 ? 4 : 2, true>(a, s);
  if (p % 4 == 0) return launch<TIn, TOut, 4, false>(a, s);
  if (p % 2 == 0) return launch<TIn, TOut, 2, false>(a, s);
  return launch<TIn, TOut, 1, false>(a, s);
}

}  // namespace

cudaError_t launch_rotary(const Geom& g, const sla_rotary& r, const i64* raw_strides, void* const* raw,
                          void* const* rot, int tensors, bool rot_f32, const int32_t* positions,
                          bool pos_batched, const int32_t* perm, bool inverse, cudaStream_t s) {
  RotaryArgs a{};
  const Side dense{i64(g.H) * g.N * g.d, i64(g.N) * g.d, g.d};
  const Side rs{raw_strides[0], raw_strides[1], raw_strides[2]};
  for (int i = 0; i < tensors; ++i) {
    a.src[i] = inverse ? rot[i] : raw[i];
    a.dst[i] = inverse ? raw[i] : rot[i];
  }
  a.in = inverse ? dense : rs;
  a.out = inverse ? rs : dense;
  a.positions = positions;
  a.perm = perm;
  a.tokens = i64(g.B) * g.N;
  a.N = g.N;
  a.H = g.H;
  a.d = g.d;
  a.tensors = tensors;
  a.pairs = r.rot_dim / 2;
  a.axes = r.axes;
  a.split1 = r.axis_pairs[0];
  a.split2 = r.axis_pairs[0] + r.axis_pairs[1];
  a.grid_r = std::max(1, r.grid[1]);
  a.grid_c = std::max(1, r.grid[2]);
  for (int i = 0; i < 3; ++i) a.origin[i] = r.origin[i];
  a.pos_batched = pos_batched;
  a.gather = !inverse;
  a.sign = inverse ? -1.f : 1.f;
  a.amplitude = r.amplitude;
  constexpr double kTurn = 0.15915494309189533577;  // 1 / 2 pi
  for (int i = 0; i < a.pairs; ++i) a.turns[i] = r.freq[i] * kTurn;
  const bool inter = r.layout == SLA_ROTARY_INTERLEAVED;
  using bf = __nv_bfloat16;
  if (g.dtype == SLA_F32) return dispatch<float, float>(a, inter, s);
  if (!rot_f32) return dispatch<bf, bf>(a, inter, s);
  return inverse ? dispatch<float, bf>(a, inter, s) : dispatch<bf, float>(a, inter, s);
}

}  // namespace sla
