// norms.hip -- the AllReduce of a block's partial products with the norms
// before and after the block, its gate and residual scale, and the gradient.
//
//   s = sum_r P_r        u = s rstd(s) w_post, or s        rstd(x) = (mean x^2 + eps)^(-1/2)
//   h = a x + g u        y_k = h rstd(h) w_pre
//
// x is the residual stream in front of the block, h the one behind it, y the
// next block's input; the gate g is one vector, or one a group of rows.  From
// the gradients of h (summed over its copies: e) and of y (summed: n), with
// r = rstd(h), q = rstd(s):
//
//   d = e + r (n w_pre - h r^2 mean(n w_pre h))        dx = a d
//   dg = sum over the group's rows of d u              v = d g
//   ds = q (v w_post - s q^2 mean(v w_post s)), or v   the same for every rank
//   dw_pre = sum over rows of n h r                    dw_post = sum over rows of v s q
//
// A workgroup takes a row at a time, its elements in registers between the
// two reductions; every stream is read and written once.  Sums are fp32, in
// an order that depends on the shapes alone; the gradient takes the statistics
// of h and s from the stored rows, which it reads anyway.
//
// Bound by memory.  Measured (kernels): forward, 4096 x 7168 bf16, 4 partials, a
// residual, a gate, 6 outputs 117 to 124 us (5.5 TB/s of 646 MB), 4096 x 4096 fp32
// 138, 1 row of 7168 6.4 us (two dependent reductions of a row over 14 waves);
// gradient, 4096 x 7168 bf16, 9 streams 121 us (4.4 TB/s) and 5 for the weights'
// sums; 104 x 2051 fp32 9.1 + 4.4; 73153 x 328 bf16 with a gate a row 98 to 102 +
// 16.  Rows of more than a vector a thread (8192 of bf16, 4096 of fp32) do not fit
// their registers and spill: gradient, 2048 x 16384 bf16 189 us + 9, 4096 x 7168
// fp32 251 to 269 + 5, 512 x 32768 fp32 631 + 17; forward, from 16385 of fp32 on
// (1024 x 32768 379).
#include "op_common.h"

namespace rar {
namespace {

constexpr int64_t kMaxRows = int64_t(1) << 24;
constexpr int64_t kMaxNormWidth = 32768;
constexpr int kMaxThreads = 1024;

__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float wave_sum(float v) {
  v = group_reduce<32>(v, add);
  return v + __shfl_xor(v, 32);
}
// The workgroup's sums of two values.  `scratch` is free again after the next
// barrier.
__device__ __forceinline__ void block_sum2(float& a, float& b, v2f* scratch, int waves) {
  a = wave_sum(a);
  b = wave_sum(b);
  if (waves == 1) return;
  if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v2f{a, b};
  __syncthreads();
  a = scratch[0][0], b = scratch[0][1];
  for (int w = 1; w < waves; ++w) a += scratch[w][0], b += scratch[w][1];
}
__device__ __forceinline__ float rstd_of(float squares, float width, float eps) { return 1.0f / __builtin_sqrtf(squares / width + eps); }

// What a row x and, for its gradient, a row v of the gradients of x / rms(x)
// are reduced to.  A row whose sum of squares leaves fp32's range is taken
// times kDown (from `scale_down` on) and summed again: no square of
// a finite number leaves it then, and what is lost at the other end is below
// 2^-60 of the row's largest element.  Where the sum of v x leaves it, v's
// part of that sum is taken times kDown.  All threads agree on both, and other
// rows see nothing of it but a comparison.
constexpr float kDown = 0x1p-80f;
struct Stats {
  float r;     // rstd of the row as it is now
  float c;     // mean(v x) r^2, likewise
  float rstd;  // of the row as it was
};
// sums(squares, dot, factor): of x^2 and of (v factor) x, over the workgroup
template <class S, class D>
__device__ __forceinline__ Stats row_stats(float width, float eps, S sums, D scale_down) {
  float squares = 0.0f, dot = 0.0f;
  sums(squares, dot, 1.0f);
  Stats s;
  s.r = s.rstd = rstd_of(squares, width, eps);
  s.c = dot / width * s.r * s.r;
  const bool in_range = s.r > 0.0f, dot_in_range = __builtin_fabsf(dot) < __builtin_inff();
  if (__builtin_expect(__ballot(!in_range || !dot_in_range) != 0, 0)) {
    const float factor = dot_in_range ? 1.0f : kDown;
    if (!in_range) scale_down();
    __syncthreads();  // the first sums have been read
    squares = dot = 0.0f;
    sums(squares, dot, factor);
    s.r = rstd_of(squares, width, in_range ? eps : eps * kDown * kDown);
    s.rstd = in_range ? s.r : s.r * kDown;
    s.c = dot / width * s.r * s.r / factor;
  }
  return s;
}

// This thread's vectors of a row: vector j starts at element (j * threads +
// threadIdx.x) * kVec.
template <class T, int kVecs>
struct Row {
  v4u v[kVecs];
  static __device__ __forceinline__ RowEdge<T> edge(int j, int width) { return RowEdge<T>((j * blockDim.x + threadIdx.x) * T::kVec, width); }
  __device__ __forceinline__ void load(const void* buf, int64_t stride, int64_t row, int width) {
    const typename T::bits* p = static_cast<const typename T::bits*>(buf) + row * stride;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) v[j] = edge(j, width).load(p);
  }
  // data that other workgroups read too
  __device__ __forceinline__ void load_shared(const void* buf, int64_t stride, int64_t row, int width) {
    const typename T::bits* p = static_cast<const typename T::bits*>(buf) + row * stride;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) v[j] = edge(j, width).load_shared(p);
  }
  // Once, between a load and the first use.
  __device__ __forceinline__ void fix(int width) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) edge(j, width).fix(v[j]);
  }
  __device__ __forceinline__ void widen(int j, float* f) const { T::widen(v[j], f); }
  __device__ __forceinline__ void set(int j, const float* f) { v[j] = T::round(f); }
  __device__ __forceinline__ void store(void* buf, int64_t stride, int64_t row, int width) const {
    typename T::bits* p = static_cast<typename T::bits*>(buf) + row * stride;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int e = (j * blockDim.x + threadIdx.x) * T::kVec;
      if (e < width) store_part<T>(p + e, width - e, v[j]);
    }
  }
};

// sum = the sum over n buffers, in order.
template <class T, int kVecs>
__device__ __forceinline__ void sum_rows(const void* const* bufs, const int64_t* strides, int n, int64_t row, int width,
                                         float (&sum)[kVecs][T::kVec]) {
  constexpr int kBatch = 4;  // buffers whose loads are issued together
#pragma unroll
  for (int j = 0; j < kVecs; ++j)
#pragma unroll
    for (int i = 0; i < T::kVec; ++i) sum[j][i] = 0.0f;
  for (int r0 = 0; r0 < n; r0 += kBatch) {
    Row<T, kVecs> x[kBatch];
#pragma unroll
    for (int r = 0; r < kBatch; ++r)
      if (r0 + r < n) x[r].load(bufs[r0 + r], strides[r0 + r], row, width);
#pragma unroll
    for (int r = 0; r < kBatch; ++r) {
      if (r0 + r < n) {
        x[r].fix(width);
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          float f[T::kVec];
          x[r].widen(j, f);
#pragma unroll
          for (int i = 0; i < T::kVec; ++i) sum[j][i] = r0 + r == 0 ? f[i] : sum[j][i] + f[i];
        }
      }
    }
  }
}

struct ForwardArgs {
  const void* src[kMaxRanks];
  int64_t src_stride[kMaxRanks];
  void* hidden[kMaxRanks];
  int64_t hidden_stride[kMaxRanks];
  void* out[kMaxRanks];
  int64_t out_stride[kMaxRanks];
  const void *residual, *post, *gate, *pre;
  void* total;
  int64_t residual_stride, total_stride, gate_stride;
  int64_t rows, group_rows;  // group_rows: rows that share a gate
  int32_t width, nsrc, nhidden, nout;
  float eps, scale;
  uint32_t block0;  // rows in earlier launches
};

// Up to two vectors a thread, two workgroups of 16 waves a CU: 2048 x 16384 bf16
// 139 us, although 12 registers spill; with none spilled and one workgroup 144.
template <class T, int kVecs>
__global__ void __launch_bounds__(kMaxThreads) __attribute__((amdgpu_waves_per_eu(kVecs <= 2 ? 8 : 4))) norms_kernel(ForwardArgs) {
  const ForwardArgs& args = kernel_args<ForwardArgs>();
  __shared__ v2f scratch[2][kMaxThreads / 64];
  const int width = args.width, waves = blockDim.x >> 6;
  const int64_t row = args.block0 + blockIdx.x;
  Row<T, kVecs> x, w, g;
  float h[kVecs][T::kVec];
  auto rstd_of_h = [&](v2f* sums) {
    return row_stats((float)width, args.eps, [&](float& squares, float& none, float) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
#pragma unroll
        for (int i = 0; i < T::kVec; ++i) squares += h[j][i] * h[j][i];
      block_sum2(squares, none, sums, waves);
    }, [&] {
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
#pragma unroll
        for (int i = 0; i < T::kVec; ++i) h[j][i] *= kDown;
    }).r;
  };
  sum_rows<T, kVecs>(args.src, args.src_stride, args.nsrc, row, width, h);
  if (args.residual) x.load(args.residual, args.residual_stride, row, width);
  if (args.total) {
    Row<T, kVecs> o;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) o.set(j, h[j]);
    o.store(args.total, args.total_stride, row, width);
  }
  if (args.gate) g.load_shared(args.gate, args.gate_stride, row / args.group_rows, width);
  if (args.post) {
    w.load_shared(args.post, 0, 0, width);
    const float q = rstd_of_h(scratch[0]);
    w.fix(width);
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      float f[T::kVec];
      w.widen(j, f);
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) h[j][i] = h[j][i] * q * f[i];
    }
  }
  if (args.gate) {
    g.fix(width);
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      float f[T::kVec];
      g.widen(j, f);
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) h[j][i] *= f[i];
    }
  }
  if (args.residual) {
    x.fix(width);
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      float f[T::kVec];
      x.widen(j, f);
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) h[j][i] += args.scale * f[i];
    }
  }
#pragma unroll
  for (int j = 0; j < kVecs; ++j) x.set(j, h[j]);
  for (int k = 0; k < args.nhidden; ++k) x.store(args.hidden[k], args.hidden_stride[k], row, width);
  if (args.nout == 0) return;
  w.load_shared(args.pre, 0, 0, width);
  const float r = rstd_of_h(scratch[1]);
  w.fix(width);
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    float f[T::kVec];
    w.widen(j, f);
#pragma unroll
    for (int i = 0; i < T::kVec; ++i) f[i] = h[j][i] * r * f[i];
    x.set(j, f);
  }
  for (int k = 0; k < args.nout; ++k) x.store(args.out[k], args.out_stride[k], row, width);
}

// ---- gradient ----------------------------------------------------------------

struct BackwardArgs {
  const void* grad_hidden[kMaxRanks];
  int64_t grad_hidden_stride[kMaxRanks];
  const void* grad_out[kMaxRanks];
  int64_t grad_out_stride[kMaxRanks];
  void* dsrc[kMaxRanks];
  int64_t dsrc_stride[kMaxRanks];
  const void *total, *hidden, *post, *gate, *pre;
  void *dresidual, *dpost, *dgate, *dpre;
  int64_t total_stride, hidden_stride, gate_stride, dresidual_stride, dgate_stride;
  float* partial;      // [workgroups][2][width]: dw_post, dw_pre; then [pieces][width]: dg
  int64_t rows, group_rows;
  int64_t pieces, piece_rows;  // runs of rows; none crosses a group
  int64_t group_pieces;        // pieces of a group
  int32_t groups;              // workgroups
  int32_t width, ngrad_hidden, ngrad_out, ndsrc;
  float eps, scale;
};

// This thread's elements of a row of sums.
template <class T, int kVecs>
__device__ __forceinline__ void store_sums(float* p, int width, const float (&sum)[kVecs][T::kVec]) {
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int e = (j * blockDim.x + threadIdx.x) * T::kVec;
#pragma unroll
    for (int i = 0; i < T::kVec; i += 4)
      if (e + i < width) store4<F32>(reinterpret_cast<uint32_t*>(p + e + i), width - e - i, sum[j] + i);
  }
}

// Workgroup b takes pieces b, b + workgroups, ...; the sums over rows stay on
// the chip: dw_pre's in registers until the workgroup ends, and of a piece the
// sum of d s q alone, from which come dg (times w_post) and dw_post (times g,
// which is the same for all rows of a piece), the latter in LDS until the
// workgroup ends.
template <class T, int kVecs>
__global__ void __launch_bounds__(kMaxThreads) norms_backward_kernel(BackwardArgs) {
  const BackwardArgs& args = kernel_args<BackwardArgs>();
  __shared__ v2f scratch[2][kMaxThreads / 64];
  __shared__ v4f dpost[T::kVec / 4 * kVecs][kMaxThreads];
  const int width = args.width, waves = blockDim.x >> 6;
  float dpre[kVecs][T::kVec], both[kVecs][T::kVec];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
#pragma unroll
    for (int i = 0; i < T::kVec; ++i) dpre[j][i] = 0.0f;
#pragma unroll
    for (int i = 0; i < T::kVec / 4; ++i) dpost[j * (T::kVec / 4) + i][threadIdx.x] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }
  const bool need_s = args.post || args.dgate;
  for (int64_t piece = blockIdx.x; piece < args.pieces; piece += args.groups) {
    const int64_t group = piece / args.group_pieces, first = (piece - group * args.group_pieces) * args.piece_rows;
    const int64_t row0 = group * args.group_rows + first;
    const int64_t row1 = group * args.group_rows + std::min(args.group_rows, first + args.piece_rows);
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) both[j][i] = 0.0f;
    for (int64_t row = row0; row < row1; ++row) {
      float d[kVecs][T::kVec];
      Row<T, kVecs> s, w, g;
      if (need_s) s.load(args.total, args.total_stride, row, width);
      sum_rows<T, kVecs>(args.grad_hidden, args.grad_hidden_stride, args.ngrad_hidden, row, width, d);
      if (args.ngrad_out) {
        Row<T, kVecs> h;
        h.load(args.hidden, args.hidden_stride, row, width);
        float n[kVecs][T::kVec];
        sum_rows<T, kVecs>(args.grad_out, args.grad_out_stride, args.ngrad_out, row, width, n);
        w.load_shared(args.pre, 0, 0, width);
        h.fix(width);
        w.fix(width);
        float down = 1.0f;  // scaling the row in its registers instead: 213 us where this takes 192 (2048 x 16384 bf16)
        const Stats of = row_stats((float)width, args.eps, [&](float& squares, float& dot, float factor) {
#pragma unroll
          for (int j = 0; j < kVecs; ++j) {
            float f[T::kVec], k[T::kVec];
            h.widen(j, f);
            w.widen(j, k);
#pragma unroll
            for (int i = 0; i < T::kVec; ++i) {
              f[i] *= down;
              squares = __builtin_fmaf(f[i], f[i], squares);
              dot = __builtin_fmaf(n[j][i] * k[i] * factor, f[i], dot);
            }
          }
          block_sum2(squares, dot, scratch[0], waves);
        }, [&] { down = kDown; });
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          float f[T::kVec], k[T::kVec];
          h.widen(j, f);
          w.widen(j, k);
#pragma unroll
          for (int i = 0; i < T::kVec; ++i) {
            f[i] *= down;
            dpre[j][i] = __builtin_fmaf(n[j][i], f[i] * of.r, dpre[j][i]);
            d[j][i] = __builtin_fmaf(of.rstd, __builtin_fmaf(-f[i], of.c, n[j][i] * k[i]), d[j][i]);
          }
        }
      }
      if (args.dresidual) {
        Row<T, kVecs> o;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          float f[T::kVec];
#pragma unroll
          for (int i = 0; i < T::kVec; ++i) f[i] = args.scale * d[j][i];
          o.set(j, f);
        }
        o.store(args.dresidual, args.dresidual_stride, row, width);
      }
      // d becomes v w_post (or v)
      if (args.gate) g.load_shared(args.gate, args.gate_stride, group, width);
      if (args.gate) g.fix(width);
      if (need_s) s.fix(width);
      if (args.post) {
        w.load_shared(args.post, 0, 0, width);
        w.fix(width);
        float down = 1.0f;
        const Stats of = row_stats((float)width, args.eps, [&](float& squares, float& dot, float factor) {
#pragma unroll
          for (int j = 0; j < kVecs; ++j) {
            float f[T::kVec], k[T::kVec], a[T::kVec];
            s.widen(j, f);
            w.widen(j, k);
            if (args.gate) g.widen(j, a);
#pragma unroll
            for (int i = 0; i < T::kVec; ++i) {
              f[i] *= down;
              squares = __builtin_fmaf(f[i], f[i], squares);
              dot = __builtin_fmaf(d[j][i] * (args.gate ? a[i] : 1.0f) * k[i] * factor, f[i], dot);
            }
          }
          block_sum2(squares, dot, scratch[1], waves);
        }, [&] { down = kDown; });
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          float f[T::kVec], k[T::kVec], a[T::kVec];
          s.widen(j, f);
          w.widen(j, k);
          if (args.gate) g.widen(j, a);
#pragma unroll
          for (int i = 0; i < T::kVec; ++i) {
            f[i] *= down;
            both[j][i] = __builtin_fmaf(d[j][i], f[i] * of.r, both[j][i]);
            d[j][i] = of.rstd * __builtin_fmaf(-f[i], of.c, d[j][i] * (args.gate ? a[i] : 1.0f) * k[i]);
          }
        }
      } else if (args.gate) {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          float f[T::kVec], a[T::kVec];
          if (args.dgate) s.widen(j, f);
          g.widen(j, a);
#pragma unroll
          for (int i = 0; i < T::kVec; ++i) {
            if (args.dgate) both[j][i] = __builtin_fmaf(d[j][i], f[i], both[j][i]);
            d[j][i] *= a[i];
          }
        }
      }
      if (args.ndsrc) {
        Row<T, kVecs> o;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) o.set(j, d[j]);
        for (int k = 0; k < args.ndsrc; ++k) o.store(args.dsrc[k], args.dsrc_stride[k], row, width);
      }
      // with several waves the barrier of one reduction frees the other's
      // scratch, unless there is only one of the two
      if ((args.ngrad_out > 0) != (args.post != nullptr) && waves > 1) __syncthreads();
    }
    if (args.dpost) {
      Row<T, kVecs> g;
      if (args.gate) g.load_shared(args.gate, args.gate_stride, group, width);
      if (args.gate) g.fix(width);
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        float a[T::kVec];
        if (args.gate) g.widen(j, a);
#pragma unroll
        for (int i = 0; i < T::kVec; ++i) dpost[(j * T::kVec + i) / 4][threadIdx.x][i % 4] += args.gate ? a[i] * both[j][i] : both[j][i];
      }
    }
    if (args.dgate) {
      if (args.post) {
        Row<T, kVecs> w;
        w.load_shared(args.post, 0, 0, width);
        w.fix(width);
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          float k[T::kVec];
          w.widen(j, k);
#pragma unroll
          for (int i = 0; i < T::kVec; ++i) both[j][i] *= k[i];
        }
      }
      if (args.group_pieces == 1) {
        Row<T, kVecs> o;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) o.set(j, both[j]);
        o.store(args.dgate, args.dgate_stride, group, width);
      } else {
        store_sums<T, kVecs>(args.partial + (2 * args.groups + piece) * width, width, both);
      }
    }
  }
  if (args.dpre) store_sums<T, kVecs>(args.partial + (2 * (int64_t)blockIdx.x + 1) * width, width, dpre);
  if (args.dpost) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) both[j][i] = dpost[(j * T::kVec + i) / 4][threadIdx.x][i % 4];
    store_sums<T, kVecs>(args.partial + 2 * (int64_t)blockIdx.x * width, width, both);
  }
}

// The same for rows of one vector a thread: the next row's loads (of total,
// hidden, a gradient of hidden and up to 4 of outs) are issued before a row is
// reduced, and none of them depends on a condition, so that the compiler's
// waits are for the row in hand alone.  An absent input is another one read
// again, and the row's end is as RowEdge has it (kEdge: it is not where a
// wave's vectors end).  Further gradients (kMore) are read where they are added.
// The row behind a piece's last is the first of the workgroup's next piece
// (73153 x 328 with a gate a row: 137 us without that, 95 to 102 with it).  16 waves of
// 128 registers a CU, so one workgroup of a wide row: without the loads ahead
// 4096 x 7168 took 151 us, with them 121 (16 rows a workgroup, each 5.5 us of
// memory and 3.3 of arithmetic, which overlap in part).
template <class T, bool kEdge, bool kMore>
__global__ void __launch_bounds__(kMaxThreads) norms_backward_ahead_kernel(BackwardArgs) {
  const BackwardArgs& args = kernel_args<BackwardArgs>();
  // gradients of outs on their way ahead, what registers hold.  4096 x 7168 bf16:
  // 4 ranks 121 us; 1 rank, where three loads read the same row again, 109; 8
  // ranks, the other four loaded when they are added, 162
  constexpr int kOuts = 4;
  typedef typename T::bits Bits;
  struct Inputs {
    v4u s, h, e, n[kOuts];
  };
  __shared__ v2f scratch[2][kMaxThreads / 64];
  // a thread's own: pre, post, gate and its part of dpost (registers are needed
  // for the rows)
  extern __shared__ v4u own_lds[];
  v4u* weights = own_lds + threadIdx.x;
  v4f* dpost = reinterpret_cast<v4f*>(own_lds + 3 * blockDim.x) + threadIdx.x;
  const int width = args.width, waves = blockDim.x >> 6;
  const int e = threadIdx.x * T::kVec, at_e = std::min(e, width - T::kVec), shift = std::min(e - at_e, T::kVec);
  const bool there = e < width;
  const int left = width - e;  // of it, more than a vector in all threads but the last
  const uint32_t at = at_e * (uint32_t)sizeof(Bits);
  // only waves with the row's end have something to shift
  const bool edge = kEdge && __ballot(shift > 0) != 0;
  auto fix = [&](v4u v) { return shift_elements<T>(v, shift); };
  auto put = [&](void* p, int64_t offset, const float* f) {
    char* row = row_at(static_cast<char*>(p), offset * (int64_t)sizeof(Bits));
    if (!kEdge || left >= T::kVec) store_nt(row + at, T::round(f));
    else if (there) store_part<T>(reinterpret_cast<Bits*>(row) + e, left, T::round(f));
  };
  const bool has_out = args.ngrad_out > 0, has_hidden = args.ngrad_hidden > 0, need_s = args.post || args.dgate;
  struct Source {
    const char* p;
    int64_t step;  // bytes
  };
  // some input that is there stands for those that are not
  const Source some = has_out ? Source{static_cast<const char*>(args.grad_out[0]), args.grad_out_stride[0]}
                              : Source{static_cast<const char*>(args.grad_hidden[0]), args.grad_hidden_stride[0]};
  auto source = [&](bool is, const void* p, int64_t stride) {
    return Source{is ? static_cast<const char*>(p) : some.p, (is ? stride : some.step) * (int64_t)sizeof(Bits)};
  };
  const Source from_s = source(need_s, args.total, args.total_stride), from_h = source(has_out, args.hidden, args.hidden_stride),
               from_e = source(has_hidden, args.grad_hidden[0], args.grad_hidden_stride[0]),
               from_n[kOuts] = {source(args.ngrad_out > 0, args.grad_out[0], args.grad_out_stride[0]),
                                source(args.ngrad_out > 1, args.grad_out[1], args.grad_out_stride[1]),
                                source(args.ngrad_out > 2, args.grad_out[2], args.grad_out_stride[2]),
                                source(args.ngrad_out > 3, args.grad_out[3], args.grad_out_stride[3])};
  auto load = [&](int64_t row, Inputs& in) {
    in.h = load_nt(row_at(from_h.p, row * from_h.step) + at);
#pragma unroll
    for (int k = 0; k < kOuts; ++k) in.n[k] = load_nt(row_at(from_n[k].p, row * from_n[k].step) + at);
    in.e = load_nt(row_at(from_e.p, row * from_e.step) + at);
    in.s = load_nt(row_at(from_s.p, row * from_s.step) + at);
  };
  // 1 for weights that are not there
  auto weight = [&](const void* p, int64_t offset) {
    float one[T::kVec];
#pragma unroll
    for (int i = 0; i < T::kVec; ++i) one[i] = 1.0f;
    const v4u v = p ? load_16(reinterpret_cast<const char*>(static_cast<const Bits*>(p) + offset) + at) : T::round(one);
    return edge ? fix(v) : v;
  };
  // sum += what the k-th and further buffers have in a row
  auto add_more = [&](const void* const* bufs, const int64_t* strides, int k, int n, int64_t row, float* sum) {
    for (; k < n; k += kOuts) {
      v4u x[kOuts];
#pragma unroll
      for (int o = 0; o < kOuts; ++o) {
        const int from = std::min(k + o, n - 1);
        x[o] = load_nt(row_at(static_cast<const char*>(bufs[from]), row * strides[from] * (int64_t)sizeof(Bits)) + at);
      }
#pragma unroll
      for (int o = 0; o < kOuts; ++o) {
        float f[T::kVec];
        T::widen(edge ? fix(x[o]) : x[o], f);
#pragma unroll
        for (int i = 0; i < T::kVec; ++i) sum[i] = k + o < n ? sum[i] + f[i] : sum[i];
      }
    }
  };
  weights[0] = weight(has_out ? args.pre : nullptr, 0);
  weights[blockDim.x] = weight(args.post, 0);
  float dpre[T::kVec];
#pragma unroll
  for (int i = 0; i < T::kVec; ++i) dpre[i] = 0.0f;
#pragma unroll
  for (int i = 0; i < T::kVec / 4; ++i) dpost[i * blockDim.x] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  float both[T::kVec];
  int64_t piece = blockIdx.x, group, row, row1;  // the row in hand and its piece's end
  auto begin_piece = [&] {
    group = piece / args.group_pieces;
    const int64_t first = (piece - group * args.group_pieces) * args.piece_rows;
    row = group * args.group_rows + first;
    row1 = group * args.group_rows + std::min(args.group_rows, first + args.piece_rows);
    weights[2 * blockDim.x] = weight(args.gate, group * args.gate_stride);
#pragma unroll
    for (int i = 0; i < T::kVec; ++i) both[i] = 0.0f;
  };
  // the row behind this one, of this piece or the workgroup's next; or itself
  auto next_row = [&] {
    if (row + 1 < row1) return row + 1;
    const int64_t next = piece + args.groups;
    if (next >= args.pieces) return row;
    const int64_t g = next / args.group_pieces;
    return g * args.group_rows + (next - g * args.group_pieces) * args.piece_rows;
  };
  auto one_row = [&](Inputs& now, Inputs& ahead) {
    float more[T::kVec];  // of the gradients of outs
    if (kMore && args.ngrad_out > kOuts) {
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) more[i] = 0.0f;
      add_more(args.grad_out, args.grad_out_stride, kOuts, args.ngrad_out, row, more);
    }
    load(next_row(), ahead);
    __builtin_amdgcn_sched_barrier(0);
    if (edge) {
      now.s = fix(now.s), now.h = fix(now.h), now.e = fix(now.e);
#pragma unroll
      for (int k = 0; k < kOuts; ++k) now.n[k] = fix(now.n[k]);
    }
    float d[T::kVec], g[T::kVec];
    if (has_out) {
      float n[T::kVec], f[T::kVec], k[T::kVec];
      T::widen(now.n[0], n);
#pragma unroll
      for (int o = 1; o < kOuts; ++o) {
        float x[T::kVec];
        T::widen(now.n[o], x);
#pragma unroll
        for (int i = 0; i < T::kVec; ++i) n[i] = o < args.ngrad_out ? n[i] + x[i] : n[i];
      }
      __builtin_amdgcn_sched_barrier(0);
      if (kMore && args.ngrad_out > kOuts) {
#pragma unroll
        for (int i = 0; i < T::kVec; ++i) n[i] += more[i];
      }
      T::widen(now.h, f);
      T::widen(weights[0], k);
      const Stats of = row_stats((float)width, args.eps, [&](float& squares, float& dot, float factor) {
#pragma unroll
        for (int i = 0; i < T::kVec; ++i) {
          squares = __builtin_fmaf(f[i], f[i], squares);
          dot = __builtin_fmaf(n[i] * k[i] * factor, f[i], dot);
        }
        block_sum2(squares, dot, scratch[0], waves);
      }, [&] {
#pragma unroll
        for (int i = 0; i < T::kVec; ++i) f[i] *= kDown;
      });
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) {
        dpre[i] = __builtin_fmaf(n[i], f[i] * of.r, dpre[i]);
        n[i] = __builtin_fmaf(-f[i], of.c, n[i] * k[i]);
      }
      T::widen(now.e, d);
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) d[i] = has_hidden ? d[i] : 0.0f;
      if (kMore && args.ngrad_hidden > 1) add_more(args.grad_hidden, args.grad_hidden_stride, 1, args.ngrad_hidden, row, d);
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) d[i] = __builtin_fmaf(of.rstd, n[i], d[i]);
    } else {
      T::widen(now.e, d);
      if (kMore && args.ngrad_hidden > 1) add_more(args.grad_hidden, args.grad_hidden_stride, 1, args.ngrad_hidden, row, d);
    }
    if (args.dresidual) {
      float f[T::kVec];
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) f[i] = args.scale * d[i];
      put(args.dresidual, row * args.dresidual_stride, f);
    }
    T::widen(weights[2 * blockDim.x], g);
    float f[T::kVec];
    T::widen(now.s, f);
    if (args.post) {
      float k[T::kVec];
      T::widen(weights[blockDim.x], k);
      const Stats of = row_stats((float)width, args.eps, [&](float& squares, float& dot, float factor) {
#pragma unroll
        for (int i = 0; i < T::kVec; ++i) {
          squares = __builtin_fmaf(f[i], f[i], squares);
          dot = __builtin_fmaf(d[i] * g[i] * k[i] * factor, f[i], dot);
        }
        block_sum2(squares, dot, scratch[1], waves);
      }, [&] {
#pragma unroll
        for (int i = 0; i < T::kVec; ++i) f[i] *= kDown;
      });
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) {
        both[i] = __builtin_fmaf(d[i], f[i] * of.r, both[i]);
        d[i] = of.rstd * __builtin_fmaf(-f[i], of.c, d[i] * g[i] * k[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) {
        both[i] = __builtin_fmaf(d[i], f[i], both[i]);
        d[i] *= g[i];
      }
    }
    for (int k = 0; k < args.ndsrc; ++k) put(args.dsrc[k], row * args.dsrc_stride[k], d);
    // with several waves the barrier of one reduction frees the other's
    // scratch, unless there is only one of the two
    if (has_out != (args.post != nullptr) && waves > 1) __syncthreads();
  };
  // The sums of a piece that has ended.
  auto end_piece = [&] {
    if (!there) return;
    if (args.dpost) {
      float g[T::kVec];
      T::widen(weights[2 * blockDim.x], g);
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) dpost[i / 4 * blockDim.x][i % 4] += g[i] * both[i];
    }
    if (args.dgate) {
      float k[T::kVec];
      T::widen(weights[blockDim.x], k);
#pragma unroll
      for (int i = 0; i < T::kVec; ++i) both[i] *= k[i];
      if (args.group_pieces == 1) {
        put(args.dgate, group * args.dgate_stride, both);
      } else {
        float* p = args.partial + (2 * args.groups + piece) * width + e;
#pragma unroll
        for (int i = 0; i < T::kVec; i += 4) store4<F32>(reinterpret_cast<uint32_t*>(p + i), left - i, both + i);
      }
    }
  };
  // The next row is the one in hand; false: there is none.
  auto advance = [&] {
    if (++row < row1) return true;
    end_piece();
    piece += args.groups;
    if (piece >= args.pieces) return false;
    begin_piece();
    return true;
  };
  Inputs in[2];
  begin_piece();
  load(row, in[0]);
  for (;;) {
    one_row(in[0], in[1]);
    if (!advance()) break;
    one_row(in[1], in[0]);
    if (!advance()) break;
  }
  if (!there) return;
  float* p = args.partial + 2 * (int64_t)blockIdx.x * width + e;
#pragma unroll
  for (int i = 0; i < T::kVec; i += 4) {
    if (args.dpre) store4<F32>(reinterpret_cast<uint32_t*>(p + width + i), left - i, dpre + i);
    float f[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = dpost[i / 4 * blockDim.x][k];
    if (args.dpost) store4<F32>(reinterpret_cast<uint32_t*>(p + i), left - i, f);
  }
}

// Adds up the partial sums: of the weights (y = 0, 1) over the workgroups, of
// gate y - 2 over its pieces.  A workgroup takes 64 columns; each of its 16
// waves a run of the parts.
template <class T>
__global__ void __launch_bounds__(1024) norms_join_kernel(BackwardArgs) {
  const BackwardArgs& args = kernel_args<BackwardArgs>();
  __shared__ float parts[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t y = blockIdx.y, column = blockIdx.x * 64 + lane;
  const float* p;
  int64_t n, step;
  typename T::bits* out;
  if (y < 2) {
    out = static_cast<typename T::bits*>(y == 0 ? args.dpost : args.dpre);
    if (!out) return;
    p = args.partial + y * args.width;
    step = 2 * args.width;
    n = args.groups;
  } else {
    const int64_t group = y - 2;
    out = static_cast<typename T::bits*>(args.dgate) + group * args.dgate_stride;
    p = args.partial + (2 * args.groups + group * args.group_pieces) * args.width;
    step = args.width;
    n = args.group_pieces;
  }
  const int64_t each = (n + 15) / 16, begin = wave * each, end = std::min(n, begin + each);
  float sum = 0.0f;
  if (column < args.width) {
#pragma unroll 8
    for (int64_t i = begin; i < end; ++i) sum += p[i * step + column];
  }
  parts[wave][lane] = sum;
  __syncthreads();
  if (wave > 0 || column >= args.width) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) sum += parts[w][lane];
  out[column] = T::round1(sum);
}

// ---- host --------------------------------------------------------------------

struct Launch {
  int vecs, threads;
};
// Vectors a thread and threads of a row.
Launch launch_of(int64_t width, int dtype) {
  const int64_t vectors = (width + (dtype == kFloat32 ? 4 : 8) - 1) / (dtype == kFloat32 ? 4 : 8);
  Launch l{1, 0};
  while (l.vecs < 8 && (vectors + l.vecs - 1) / l.vecs > 1024) l.vecs *= 2;
  l.threads = (int)(((vectors + l.vecs - 1) / l.vecs + 63) / 64 * 64);
  return l;
}

template <class T>
const void* norm_kernel(int vecs, bool backward) {
  constexpr int kMost = (int)(kMaxNormWidth / (kMaxThreads * T::kVec));  // 4 in bf16, 8 in fp32
  if (vecs == 1) return backward ? reinterpret_cast<const void*>(&norms_backward_kernel<T, 1>) : reinterpret_cast<const void*>(&norms_kernel<T, 1>);
  if (vecs == 2) return backward ? reinterpret_cast<const void*>(&norms_backward_kernel<T, 2>) : reinterpret_cast<const void*>(&norms_kernel<T, 2>);
  if (vecs == 4) return backward ? reinterpret_cast<const void*>(&norms_backward_kernel<T, 4>) : reinterpret_cast<const void*>(&norms_kernel<T, 4>);
  return backward ? reinterpret_cast<const void*>(&norms_backward_kernel<T, kMost>) : reinterpret_cast<const void*>(&norms_kernel<T, kMost>);
}

template <class T>
const void* ahead_kernel(bool edge, bool more) {
  if (edge) return more ? reinterpret_cast<const void*>(&norms_backward_ahead_kernel<T, true, true>) : reinterpret_cast<const void*>(&norms_backward_ahead_kernel<T, true, false>);
  return more ? reinterpret_cast<const void*>(&norms_backward_ahead_kernel<T, false, true>) : reinterpret_cast<const void*>(&norms_backward_ahead_kernel<T, false, false>);
}

rar_result_t check_norm(const rar_norm_t* n) {
  if (!n) return set_error(RAR_INVALID_ARGUMENT, "norm is NULL");
  if (rar_result_t r = check_float_dtype(n->dtype)) return r;
  if (n->rows < 0 || n->rows > kMaxRows) return set_error(RAR_INVALID_ARGUMENT, "rows must be in [0, 2^24]");
  if (n->width < 1 || n->width > kMaxNormWidth) return set_error(RAR_INVALID_ARGUMENT, "width must be in [1, 32768]");
  if (!(n->eps > 0.0f && n->eps - n->eps == 0.0f)) return set_error(RAR_INVALID_ARGUMENT, "eps must be positive and finite");
  if (!(n->residual_scale - n->residual_scale == 0.0f)) return set_error(RAR_INVALID_ARGUMENT, "residual_scale must be finite");
  if (n->gate && (n->gate_groups < 1 || n->gate_groups > std::max<int64_t>(1, n->rows) || n->rows % n->gate_groups))
    return set_error(RAR_INVALID_ARGUMENT, "gate_groups must divide the rows");
  return RAR_SUCCESS;
}

// Pieces of the rows.
struct Pieces {
  int64_t group_rows, piece_rows, group_pieces, pieces, groups, bytes;
};
Pieces pieces_of(const rar_norm_t& n) {
  Pieces p;
  const int64_t gates = n.gate ? n.gate_groups : 1;
  p.group_rows = n.rows / gates;
  // as many workgroups as the device holds (16 waves a CU), their pieces of 8
  // rows or more where there are many
  const int waves = launch_of(n.width, n.dtype).threads / 64;
  const int64_t most = 256 * (16 / waves), least = n.rows <= 512 ? 1 : n.rows <= 1024 ? 2 : n.rows <= 8192 ? 4 : 8;
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(most / gates, p.group_rows / least));
  p.piece_rows = (p.group_rows + want - 1) / want;
  p.group_pieces = p.piece_rows ? (p.group_rows + p.piece_rows - 1) / p.piece_rows : 1;
  p.pieces = gates * p.group_pieces;
  p.groups = std::min<int64_t>(p.pieces, most);
  p.bytes = (2 * p.groups + (p.group_pieces > 1 ? p.pieces : 0)) * n.width * 4;
  return p;
}

// One operand of [rows, width] elements.
rar_result_t check_rows(const rar_norm_t& n, const void* p, int64_t& stride, const char* what) {
  const int64_t given = stride;
  if (rar_result_t e = set_stride(stride, given ? &given : nullptr, 0, n.width, n.rows, what)) return e;
  return check_pointer(p, elem_size(n.dtype), what);
}
rar_result_t check_list(const rar_norm_t& n, const void* const* ps, const int64_t* strides, int count, const void** to, int64_t* to_strides,
                        const char* what, std::vector<Block>* blocks, int in_place) {
  const int64_t es = elem_size(n.dtype);
  if (count > 0 && !ps) return argument_error(what, -1, "has a NULL array");
  for (int k = 0; k < count; ++k) {
    if (rar_result_t e = set_stride(to_strides[k], strides, k, n.width, n.rows, what)) return e;
    if (rar_result_t e = check_pointer(ps[k], es, what, k)) return e;
    to[k] = ps[k];
    blocks->push_back({ps[k], n.rows, n.width * es, to_strides[k] * es, what, in_place});
  }
  return RAR_SUCCESS;
}
// The weights and the gate, as inputs.
rar_result_t check_weights(const rar_norm_t& n, int64_t* gate_stride, std::vector<Block>* reads) {
  const int64_t es = elem_size(n.dtype), bytes = n.width * es;
  for (const void* w : {n.post_weight, n.pre_weight}) {
    if (!w) continue;
    if (rar_result_t e = check_pointer(w, es, "weight")) return e;
    reads->push_back({w, 1, bytes, bytes, "a weight"});
  }
  if (n.gate) {
    if (rar_result_t e = set_stride(*gate_stride, n.gate_stride ? &n.gate_stride : nullptr, 0, n.width, n.gate_groups, "gate stride")) return e;
    if (rar_result_t e = check_pointer(n.gate, es, "gate")) return e;
    reads->push_back({n.gate, n.gate_groups, bytes, *gate_stride * es, "gate"});
  }
  return RAR_SUCCESS;
}

rar_result_t forward(const rar_norm_t* norm, const void* const* partials, const int64_t* partial_strides, int nranks,
                     const void* residual, int64_t residual_stride, void* const* hidden, const int64_t* hidden_strides, int nhidden,
                     void* const* outs, const int64_t* out_strides, int nouts, void* total, int64_t total_stride, void* stream) {
  if (rar_result_t r = check_norm(norm)) return r;
  const rar_norm_t& n = *norm;
  if (nranks < 1 || nranks > kMaxRanks) return set_error(RAR_INVALID_ARGUMENT, "nranks must be in [1, 64]");
  if (nhidden < 0 || nhidden > kMaxRanks || nouts < 0 || nouts > kMaxRanks)
    return set_error(RAR_INVALID_ARGUMENT, "the numbers of outputs must be in [0, 64]");
  if (nhidden + nouts == 0) return set_error(RAR_INVALID_ARGUMENT, "no output is wanted");
  if (nouts > 0 && !n.pre_weight) return set_error(RAR_INVALID_ARGUMENT, "outs need pre_weight");
  if (n.rows == 0) return RAR_SUCCESS;
  ForwardArgs a{};
  const int64_t es = elem_size(n.dtype), bytes = n.width * es;
  // A thread reads its elements of a row from all inputs before it writes them.
  std::vector<Block> reads, writes;
  reads.reserve(nranks + 4);
  writes.reserve(nhidden + nouts + 1);
  if (rar_result_t r = check_list(n, partials, partial_strides, nranks, a.src, a.src_stride, "partial", &reads, kAnyOutput)) return r;
  if (residual) {
    if (rar_result_t r = check_rows(n, residual, residual_stride, "residual")) return r;
    reads.push_back({residual, n.rows, bytes, residual_stride * es, "residual", kAnyOutput});
  }
  if (rar_result_t r = check_weights(n, &a.gate_stride, &reads)) return r;
  if (rar_result_t r = check_list(n, hidden, hidden_strides, nhidden, const_cast<const void**>(a.hidden), a.hidden_stride, "hidden", &writes, kNoOutput)) return r;
  if (rar_result_t r = check_list(n, outs, out_strides, nouts, const_cast<const void**>(a.out), a.out_stride, "out", &writes, kNoOutput)) return r;
  if (total) {
    if (rar_result_t r = check_rows(n, total, total_stride, "total")) return r;
    writes.push_back({total, n.rows, bytes, total_stride * es, "total"});
  }
  if (rar_result_t r = check_blocks(reads, writes)) return r;
  a.residual = residual, a.post = n.post_weight, a.gate = n.gate, a.pre = n.pre_weight, a.total = total;
  a.residual_stride = residual_stride, a.total_stride = total_stride;
  a.rows = n.rows, a.group_rows = n.gate ? n.rows / n.gate_groups : n.rows;
  a.width = (int32_t)n.width, a.nsrc = nranks, a.nhidden = nhidden, a.nout = nouts;
  a.eps = n.eps, a.scale = n.residual_scale;
  const Launch l = launch_of(n.width, n.dtype);
  return launch_groups(n.dtype == kFloat32 ? norm_kernel<F32>(l.vecs, false) : norm_kernel<BF16>(l.vecs, false), n.rows, l.threads, &a,
                       &a.block0, stream);
}

rar_result_t backward(const rar_norm_t* norm, const void* const* grad_hidden, const int64_t* grad_hidden_strides, int ngrad_hidden,
                      const void* const* grad_outs, const int64_t* grad_out_strides, int ngrad_outs, const void* total, int64_t total_stride,
                      const void* hidden, int64_t hidden_stride, void* const* dpartials, const int64_t* dpartial_strides, int ndpartials,
                      void* dresidual, int64_t dresidual_stride, void* dpost, void* dgate, int64_t dgate_stride, void* dpre,
                      void* workspace, size_t workspace_bytes, void* stream) {
  if (rar_result_t r = check_norm(norm)) return r;
  const rar_norm_t& n = *norm;
  for (int count : {ngrad_hidden, ngrad_outs, ndpartials})
    if (count < 0 || count > kMaxRanks) return set_error(RAR_INVALID_ARGUMENT, "the numbers of gradients must be in [0, 64]");
  if (ngrad_hidden + ngrad_outs == 0) return set_error(RAR_INVALID_ARGUMENT, "no gradient is given");
  if (ngrad_outs > 0 && !n.pre_weight) return set_error(RAR_INVALID_ARGUMENT, "grad_outs need pre_weight");
  if (dpre && ngrad_outs == 0) return set_error(RAR_INVALID_ARGUMENT, "the gradient of pre_weight needs grad_outs");
  if (dpost && !n.post_weight) return set_error(RAR_INVALID_ARGUMENT, "the gradient of post_weight needs post_weight");
  if (dgate && !n.gate) return set_error(RAR_INVALID_ARGUMENT, "the gradient of the gate needs a gate");
  BackwardArgs a{};
  const int64_t es = elem_size(n.dtype), bytes = n.width * es;
  std::vector<Block> reads, writes;
  reads.reserve(ngrad_hidden + ngrad_outs + 5);
  writes.reserve(ndpartials + 5);
  const Pieces p = pieces_of(n);
  if (n.rows > 0) {
    if (rar_result_t r = check_list(n, grad_hidden, grad_hidden_strides, ngrad_hidden, a.grad_hidden, a.grad_hidden_stride, "grad_hidden", &reads, kAnyOutput)) return r;
    if (rar_result_t r = check_list(n, grad_outs, grad_out_strides, ngrad_outs, a.grad_out, a.grad_out_stride, "grad_out", &reads, kAnyOutput)) return r;
    if (n.post_weight || dgate) {
      if (rar_result_t r = check_rows(n, total, total_stride, "total")) return r;
      reads.push_back({total, n.rows, bytes, total_stride * es, "total", kAnyOutput});
    }
    if (ngrad_outs > 0) {
      if (rar_result_t r = check_rows(n, hidden, hidden_stride, "hidden")) return r;
      reads.push_back({hidden, n.rows, bytes, hidden_stride * es, "hidden", kAnyOutput});
    }
    if (rar_result_t r = check_list(n, dpartials, dpartial_strides, ndpartials, const_cast<const void**>(a.dsrc), a.dsrc_stride, "dpartial", &writes, kNoOutput)) return r;
    if (dresidual) {
      if (rar_result_t r = check_rows(n, dresidual, dresidual_stride, "dresidual")) return r;
      writes.push_back({dresidual, n.rows, bytes, dresidual_stride * es, "dresidual"});
    }
    if (p.bytes) {
      if (rar_result_t r = check_pointer(workspace, 1, "workspace")) return r;
      if (reinterpret_cast<uintptr_t>(workspace) & 15) return set_error(RAR_INVALID_ARGUMENT, "workspace is not aligned to 16 bytes");
      if (workspace_bytes < (size_t)p.bytes) return set_error(RAR_INVALID_ARGUMENT, "workspace is too small");
    }
  }
  if (rar_result_t r = check_weights(n, &a.gate_stride, &reads)) return r;
  // What a whole row or column is read for is no place for an element's result.
  const size_t rows_written = writes.size();
  for (void* d : {dpost, dpre}) {
    if (!d) continue;
    if (rar_result_t r = check_pointer(d, es, "the gradient of a weight")) return r;
    writes.push_back({d, 1, bytes, bytes, "the gradient of a weight"});
  }
  if (dgate) {
    if (rar_result_t r = set_stride(a.dgate_stride, dgate_stride ? &dgate_stride : nullptr, 0, n.width, n.gate_groups, "dgate stride")) return r;
    if (rar_result_t r = check_pointer(dgate, es, "the gradient of the gate")) return r;
    writes.push_back({dgate, n.gate_groups, bytes, a.dgate_stride * es, "the gradient of the gate"});
  }
  if (n.rows > 0 && p.bytes) writes.push_back({workspace, 1, p.bytes, p.bytes, "workspace"});
  for (size_t i = rows_written; i < writes.size(); ++i)
    for (const Block& r : reads)
      if (blocks_overlap(writes[i], r)) return set_error(RAR_INVALID_ARGUMENT, std::string(writes[i].what) + " overlaps " + r.what);
  if (rar_result_t r = check_blocks(reads, writes)) return r;
  a.total = total, a.hidden = hidden, a.post = n.post_weight, a.gate = n.gate, a.pre = n.pre_weight;
  a.dresidual = dresidual, a.dpost = dpost, a.dgate = dgate, a.dpre = dpre;
  a.total_stride = total_stride, a.hidden_stride = hidden_stride, a.dresidual_stride = dresidual_stride;
  a.partial = static_cast<float*>(workspace);
  a.rows = n.rows, a.group_rows = p.group_rows;
  a.pieces = n.rows ? p.pieces : 0, a.piece_rows = p.piece_rows, a.group_pieces = p.group_pieces, a.groups = n.rows ? (int32_t)p.groups : 0;
  a.width = (int32_t)n.width, a.ngrad_hidden = ngrad_hidden, a.ngrad_out = ngrad_outs, a.ndsrc = ndpartials;
  a.eps = n.eps, a.scale = n.residual_scale;
  if (n.rows > 0) {
    const Launch l = launch_of(n.width, n.dtype);
    const bool f32 = n.dtype == kFloat32;
    const bool ahead = l.vecs == 1 && n.width >= (f32 ? F32::kVec : BF16::kVec);
    const void* fn = f32 ? norm_kernel<F32>(l.vecs, true) : norm_kernel<BF16>(l.vecs, true);
    if (ahead) {
      const bool edge = n.width % (64 * (f32 ? F32::kVec : BF16::kVec)) != 0, more = ngrad_outs > 4 || ngrad_hidden > 1;
      fn = f32 ? ahead_kernel<F32>(edge, more) : ahead_kernel<BF16>(edge, more);
    }
    const unsigned lds = ahead ? l.threads * (unsigned)(3 + (f32 ? F32::kVec : BF16::kVec) / 4) * 16 : 0;
    if (rar_result_t r = launch_kernel(fn,
                                       dim3((unsigned)p.groups), dim3(l.threads), &a, stream, lds)) return r;
  }
  // Without rows the sums over them are zero, the join's over no parts.
  const bool join_gate = dgate && (n.rows == 0 || p.group_pieces > 1);
  if (!dpost && !dpre && !join_gate) return RAR_SUCCESS;
  const dim3 grid((unsigned)((n.width + 63) / 64), (unsigned)(join_gate ? 2 + n.gate_groups : 2));
  if (n.rows == 0) a.group_pieces = 0;
  return launch_kernel(n.dtype == kFloat32 ? reinterpret_cast<const void*>(&norms_join_kernel<F32>) : reinterpret_cast<const void*>(&norms_join_kernel<BF16>),
                       grid, dim3(1024), &a, stream);
}

}  // namespace
}  // namespace rar

extern "C" {

rar_result_t rar_norm_allreduce(const rar_norm_t* norm, const void* const* partials, const int64_t* partial_strides, int nranks,
                                const void* residual, int64_t residual_stride, void* const* hidden, const int64_t* hidden_strides,
                                int nhidden, void* const* outs, const int64_t* out_strides, int nouts, void* total,
                                int64_t total_stride, void* stream) {
  return rar::guarded([&] {
    return rar::forward(norm, partials, partial_strides, nranks, residual, residual_stride, hidden, hidden_strides, nhidden, outs,
                        out_strides, nouts, total, total_stride, stream);
  });
}

rar_result_t rar_norm_allreduce_backward(const rar_norm_t* norm, const void* const* grad_hidden, const int64_t* grad_hidden_strides,
                                         int ngrad_hidden, const void* const* grad_outs, const int64_t* grad_out_strides,
                                         int ngrad_outs, const void* total, int64_t total_stride, const void* hidden,
                                         int64_t hidden_stride, void* const* dpartials, const int64_t* dpartial_strides,
                                         int ndpartials, void* dresidual, int64_t dresidual_stride, void* dpost_weight, void* dgate,
                                         int64_t dgate_stride, void* dpre_weight, void* workspace, size_t workspace_bytes,
                                         void* stream) {
  return rar::guarded([&] {
    return rar::backward(norm, grad_hidden, grad_hidden_strides, ngrad_hidden, grad_outs, grad_out_strides, ngrad_outs, total,
                         total_stride, hidden, hidden_stride, dpartials, dpartial_strides, ndpartials, dresidual, dresidual_stride,
                         dpost_weight, dgate, dgate_stride, dpre_weight, workspace, workspace_bytes, stream);
  });
}

rar_result_t rar_norm_workspace(const rar_norm_t* norm, size_t* bytes) {
  return rar::guarded([&]() -> rar_result_t {
    if (!bytes) return rar::set_error(RAR_INVALID_ARGUMENT, "bytes is NULL");
    if (rar_result_t r = rar::check_norm(norm)) return r;
    *bytes = norm->rows ? (size_t)rar::pieces_of(*norm).bytes : 0;
    return RAR_SUCCESS;
  });
}

}  // extern "C"
