// adapters.hip -- low-rank adapters of many requests beside a row-parallel
// projection, with the projection's one-shot AllReduce.
//
//   y_t = sum_r P_r[t] + scale_a * B_a (sum_r A_{a,r} x_r[t]),   a = ids[t]
//
// Rank r holds the columns x_r of the input, the partial product P_r of the
// shared projection and its part A_{a,r} of each adapter; tokens with an id
// outside [0, adapters) have no adapter.  Two kernels: `shrink` forms
// h_t = A x_t in fp32, the inner dimension cut into parts over workgroups,
// and `expand` adds up the parts, forms B h, folds the ranks' partials in
// rank order and writes y to every copy, rounded to the payload type once.
//
// Both products are MFMA tiles of 16 x 16.  A tile's tokens may have different
// adapters: the adapters of a tile are taken in turn, with the other tokens'
// rows left out.  An adapter's non-finite weights reach its own tokens only.
// In bf16, h enters expand as the sum of two bf16 numbers (16 bits of it).
//
// Bound by memory: x, the partials and y move once; 2 * rank flops for each
// element of x and y are far below the matrix rate.
#include "op_common.h"

namespace rar {
namespace {

constexpr int kMaxRank = 128;  // of an adapter
constexpr int kThreads = 256, kWaves = kThreads / kWaveSize;

struct ShrinkArgs {
  const void* x[kMaxRanks];
  int64_t x_stride[kMaxRanks];
  const void* down[kMaxRanks];   // [adapters][rank][width]
  int32_t width[kMaxRanks];
  int32_t part0[kMaxRanks + 1];  // first part of each rank
  const int64_t* ids;
  float* h;                      // [parts][tokens][rank]
  int64_t tokens;
  int32_t nranks, adapters, rank, part_width, slots;
};
struct ExpandArgs {
  const void* partial[kMaxRanks];
  int64_t partial_stride[kMaxRanks];
  void* out[kMaxRanks];
  int64_t out_stride[kMaxRanks];
  const void* up;                // [adapters][outer][rank]
  const int64_t* ids;
  const float* scales;
  const float* h;
  int64_t tokens;
  int32_t nranks, ncopies, adapters, rank, outer, parts;
  int32_t tiles_per_block;       // token tiles that a workgroup takes in turn
};

// One 16-byte vector of each operand: 32 (bf16) or 16 (fp32) of the inner
// dimension, lane group g = lane / 16 holding places g * kVec ...
template <class T>
__device__ __forceinline__ v4f mma(v4u a, v4u b, v4f c) {
  if constexpr (T::kVec == 8) {
    typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0, 0, 0);
    return c;
  }
}

// The adapter of the token that this lane's copy of a tile stands for, or -1.
__device__ __forceinline__ int load_id(const int64_t* ids, int64_t token, int64_t tokens, int adapters) {
  if (token >= tokens) return -1;
  const int64_t id = ids[token];
  return id >= 0 && id < adapters ? (int)id : -1;
}

// h of 16 tokens and one part of the inner dimension, for the adapters
// slot, slot + slots, ... of the tile.  The waves split the part between them
// and their sums meet in LDS.
template <class T, int kN>  // kN tiles of 16 cover the adapter's rank
__global__ void __launch_bounds__(kThreads) shrink_kernel(ShrinkArgs) {
  const ShrinkArgs& args = kernel_args<ShrinkArgs>();
  __shared__ v4f sums[kWaves][kN][kWaveSize];
  constexpr int kStep = 4 * T::kVec;  // inner places of one vector over the lane groups
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, group = lane >> 4, at = lane & 15;
  const int64_t token0 = (int64_t)blockIdx.x * 16;
  const int part = blockIdx.y;
  int r = 0;
  while (r + 1 < args.nranks && args.part0[r + 1] <= part) ++r;
  const int width = args.width[r];
  const int begin = (part - args.part0[r]) * args.part_width;
  const int end = begin + args.part_width < width ? begin + args.part_width : width;
  const int id = load_id(args.ids, token0 + at, args.tokens, args.adapters);
  const typename T::bits* xrow =
      static_cast<const typename T::bits*>(args.x[r]) + (token0 + at) * args.x_stride[r];
  uint64_t left = __ballot(id >= 0) & 0xFFFF;
  for (int k = 0; left; ++k) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    const bool mine = id == a;
    left &= ~__ballot(mine);
    if (k % args.slots != (int)blockIdx.z) continue;
    const typename T::bits* w =
        static_cast<const typename T::bits*>(args.down[r]) + (int64_t)a * args.rank * width;
    v4f acc[kN];
#pragma unroll
    for (int n = 0; n < kN; ++n) acc[n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = begin + wave * 2 * kStep; c < end; c += kWaves * 2 * kStep) {
      // two vectors a lane, side by side: the inner dimension's order within
      // a step is free as long as both operands take the same
      v4u xa[2], wb[kN][2];
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int col = c + (group * 2 + v) * T::kVec;
        xa[v] = load_part<T>(xrow + col, mine ? end - col : 0, 0);
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          const int row = n * 16 + at;
          wb[n][v] = load_part<T>(w + (int64_t)row * width + col, row < args.rank ? end - col : 0, 0);
        }
      }
#pragma unroll
      for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int n = 0; n < kN; ++n) acc[n] = mma<T>(xa[v], wb[n][v], acc[n]);
    }
    __syncthreads();  // the previous adapter's sums have been read
#pragma unroll
    for (int n = 0; n < kN; ++n) sums[wave][n][lane] = acc[n];
    __syncthreads();
    // lane: column (place in the adapter's rank) `at`, rows (tokens) 4 * group + i
    for (int n = wave; n < kN; n += kWaves) {
      v4f s = sums[0][n][lane];
#pragma unroll
      for (int o = 1; o < kWaves; ++o) s += sums[o][n][lane];
      const int col = n * 16 + at;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * group + i;
        const int id_of_row = __builtin_amdgcn_ds_bpermute(row * 4, id);  // with every lane active
        if (col < args.rank && id_of_row == a)
          args.h[((int64_t)part * args.tokens + token0 + row) * args.rank + col] = s[i];
      }
    }
  }
}

// y of 16 tokens x 64 columns a wave, for `tiles_per_block` token tiles in
// turn.  The columns are the MFMA's rows: row m of tile j is column
// (m / 4) * 16 + j * 4 + m % 4, so that a lane's results over the four tiles
// are 16 neighbouring columns of one token.
template <class T, int kR>  // kR vectors of each lane group cover the adapter's rank
__global__ void __launch_bounds__(kThreads) expand_kernel(ExpandArgs) {
  const ExpandArgs& args = kernel_args<ExpandArgs>();
  constexpr int kStep = 4 * T::kVec, kVecs = 16 / T::kVec, kBatch = 4;
  typedef typename T::bits bits;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, group = lane >> 4, at = lane & 15;
  const int col0 = ((int)blockIdx.x * kWaves + wave) * 64;
  const int col = col0 + group * 16;
  if (col0 >= args.outer) return;
  int held = -1;  // the adapter whose weights are in registers
  v4u w[4][kR];
  for (int tile = 0; tile < args.tiles_per_block; ++tile) {
    const int64_t token0 = ((int64_t)blockIdx.y * args.tiles_per_block + tile) * 16;
    if (token0 >= args.tokens) return;
    const int64_t token = token0 + at;
    const int id = load_id(args.ids, token, args.tokens, args.adapters);
    v4f sum[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    uint64_t left = __ballot(id >= 0) & 0xFFFF;
    while (left) {
      const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
      const bool mine = id == a;
      left &= ~__ballot(mine);
      if (a != held) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int d = col0 + (at >> 2) * 16 + j * 4 + (at & 3);
          const bits* row = static_cast<const bits*>(args.up) + ((int64_t)a * args.outer + d) * args.rank;
#pragma unroll
          for (int c = 0; c < kR; ++c) {
            const int q = c * kStep + group * T::kVec;
            w[j][c] = load_part<T>(row + q, d < args.outer ? args.rank - q : 0, 0);
          }
        }
        held = a;
      }
      const float scale = args.scales ? args.scales[a] : 1.0f;
      v4f acc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < kR; ++c) {
        const int q = c * kStep + group * T::kVec;
        float h[T::kVec];
#pragma unroll
        for (int i = 0; i < T::kVec; ++i) h[i] = 0.0f;
        if (mine) {
          for (int p = 0; p < args.parts; ++p) {
            const float* src = args.h + ((int64_t)p * args.tokens + token) * args.rank + q;
#pragma unroll
            for (int i = 0; i < T::kVec; ++i)
              if (q + i < args.rank) h[i] += src[i];
          }
#pragma unroll
          for (int i = 0; i < T::kVec; ++i) h[i] *= scale;
        }
        const v4u high = T::round(h);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = mma<T>(w[j][c], high, acc[j]);
        if constexpr (T::kVec == 8) {
          float back[8];
          T::widen(high, back);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[i] -= back[i];
          const v4u low = T::round(h);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] = mma<T>(w[j][c], low, acc[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] = mine ? acc[j] : sum[j];
    }
    if (token >= args.tokens) continue;
    float y[16];
    for (int r0 = 0; r0 < args.nranks; r0 += kBatch) {
      v4u p[kBatch][kVecs];
#pragma unroll
      for (int r = 0; r < kBatch; ++r) {
        if (r0 + r < args.nranks) {
          const bits* src = static_cast<const bits*>(args.partial[r0 + r]) + token * args.partial_stride[r0 + r] + col;
#pragma unroll
          for (int v = 0; v < kVecs; ++v) p[r][v] = load_part<T>(src + v * T::kVec, args.outer - col - v * T::kVec, 0);
        }
      }
#pragma unroll
      for (int r = 0; r < kBatch; ++r) {
        if (r0 + r < args.nranks) {
          float f[16];
#pragma unroll
          for (int v = 0; v < kVecs; ++v) T::widen(p[r][v], f + v * T::kVec);
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = r0 + r == 0 ? f[i] : y[i] + f[i];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] += sum[i / 4][i % 4];
    for (int k = 0; k < args.ncopies; ++k) {
      bits* dst = static_cast<bits*>(args.out[k]) + token * args.out_stride[k] + col;
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
        store_part<T>(dst + v * T::kVec, args.outer - col - v * T::kVec, T::round(y + v * T::kVec));
    }
  }
}

template <class T>
const void* pick_shrink(int rank) {
  if (rank <= 16) return reinterpret_cast<const void*>(&shrink_kernel<T, 1>);
  if (rank <= 32) return reinterpret_cast<const void*>(&shrink_kernel<T, 2>);
  if (rank <= 64) return reinterpret_cast<const void*>(&shrink_kernel<T, 4>);
  return reinterpret_cast<const void*>(&shrink_kernel<T, 8>);
}
template <class T>
const void* pick_expand(int rank) {
  if (rank <= 4 * T::kVec) return reinterpret_cast<const void*>(&expand_kernel<T, 1>);
  if (rank <= 8 * T::kVec) return reinterpret_cast<const void*>(&expand_kernel<T, 2>);
  if (rank <= 16 * T::kVec) return reinterpret_cast<const void*>(&expand_kernel<T, 4>);
  return reinterpret_cast<const void*>(&expand_kernel<T, 8>);
}

// How the inner dimension is cut: parts of `width` that do not cross ranks.
struct Parts {
  int width = 0;
  int first[kMaxRanks + 1] = {};
};
Parts cut_parts(const int64_t* widths, int nranks, int64_t tokens, int dtype) {
  Parts p;
  int64_t inner = 0;
  for (int r = 0; r < nranks; ++r) inner += widths[r];
  // Workgroups for every compute unit twice over, no part below one step of
  // the four waves, and few parts: expand reads each part's h again.
  const int64_t tiles = std::max<int64_t>(1, (tokens + 15) / 16);
  const int64_t least = kWaves * 8 * (16 / elem_size(dtype));
  const int64_t want = std::max<int64_t>(1, 512 / tiles);
  p.width = (int)std::max<int64_t>(least, ((inner + want - 1) / want + least - 1) / least * least);
  for (int r = 0; r < nranks; ++r) p.first[r + 1] = p.first[r] + (int)((widths[r] + p.width - 1) / p.width);
  return p;
}

rar_result_t check_adapters(const int64_t* widths, int nranks, int64_t tokens, int dtype, int64_t adapters, int rank) {
  if (nranks < 1 || nranks > kMaxRanks) return set_error(RAR_INVALID_ARGUMENT, "nranks must be in [1, 64]");
  if (rar_result_t r = check_float_dtype(dtype)) return r;
  if (!widths) return set_error(RAR_INVALID_ARGUMENT, "widths is NULL");
  if (tokens < 0 || tokens > (int64_t(1) << 24)) return set_error(RAR_INVALID_ARGUMENT, "tokens must be in [0, 2^24]");
  if (adapters < 1 || adapters > (int64_t(1) << 24))
    return set_error(RAR_INVALID_ARGUMENT, "adapters must be in [1, 2^24]");
  if (rank < 1 || rank > kMaxRank) return set_error(RAR_INVALID_ARGUMENT, "the adapters' rank must be in [1, 128]");
  for (int r = 0; r < nranks; ++r)
    if (widths[r] < 0 || widths[r] > (int64_t(1) << 24))
      return set_error(RAR_INVALID_ARGUMENT, "width of rank " + std::to_string(r) + " must be in [0, 2^24]");
  return RAR_SUCCESS;
}

rar_result_t adapter_call(const void* const* xs, const int64_t* widths, const int64_t* x_strides,
                          const void* const* partials, const int64_t* partial_strides, int nranks, void* const* outs,
                          const int64_t* out_strides, int ncopies, int64_t tokens, int64_t outer, int dtype,
                          const void* const* downs, const void* up, int64_t adapters, int rank, const int64_t* ids,
                          const float* scales, void* workspace, size_t workspace_bytes, void* stream) {
  if (rar_result_t r = check_adapters(widths, nranks, tokens, dtype, adapters, rank)) return r;
  if (ncopies < 1 || ncopies > kMaxRanks) return set_error(RAR_INVALID_ARGUMENT, "the number of copies must be in [1, 64]");
  if (outer < 1 || outer > (int64_t(1) << 24)) return set_error(RAR_INVALID_ARGUMENT, "outer must be in [1, 2^24]");
  if (tokens == 0) return RAR_SUCCESS;
  if (!xs || !partials || !outs || !downs) return set_error(RAR_INVALID_ARGUMENT, "an array of buffers is NULL");
  const size_t es = (size_t)elem_size(dtype);
  ShrinkArgs s{};
  ExpandArgs e{};
  std::vector<Block> reads, partial_reads, writes, scratch;
  auto flat = [](const void* p, int64_t bytes, const char* what) { return Block{p, 1, bytes, bytes, what}; };
  for (int r = 0; r < nranks; ++r) {
    const std::string of = " of rank " + std::to_string(r);
    s.width[r] = (int32_t)widths[r];
    s.x_stride[r] = x_strides ? x_strides[r] : widths[r];
    if (s.x_stride[r] < widths[r]) return set_error(RAR_INVALID_ARGUMENT, "input row stride" + of + " below its width");
    if (widths[r]) {
      if (rar_result_t q = check_pointer(xs[r], es, "input" + of)) return q;
      if (rar_result_t q = check_pointer(downs[r], es, "down weights" + of)) return q;
      reads.push_back({xs[r], tokens, (int64_t)(widths[r] * es), (int64_t)(s.x_stride[r] * es), "an input"});
      reads.push_back(flat(downs[r], adapters * rank * widths[r] * (int64_t)es, "down weights"));
    }
    s.x[r] = xs[r];
    s.down[r] = downs[r];
    e.partial_stride[r] = partial_strides ? partial_strides[r] : outer;
    if (e.partial_stride[r] < outer) return set_error(RAR_INVALID_ARGUMENT, "partial row stride" + of + " below its width");
    if (rar_result_t q = check_pointer(partials[r], es, "partial" + of)) return q;
    e.partial[r] = partials[r];
    partial_reads.push_back({partials[r], tokens, (int64_t)(outer * es), (int64_t)(e.partial_stride[r] * es), "a partial"});
  }
  for (int k = 0; k < ncopies; ++k) {
    e.out_stride[k] = out_strides ? out_strides[k] : outer;
    if (e.out_stride[k] < outer)
      return set_error(RAR_INVALID_ARGUMENT, "output row stride " + std::to_string(k) + " below its width");
    if (rar_result_t q = check_pointer(outs[k], es, "output " + std::to_string(k))) return q;
    e.out[k] = outs[k];
    writes.push_back({outs[k], tokens, (int64_t)(outer * es), (int64_t)(e.out_stride[k] * es), "output"});
  }
  if (rar_result_t q = check_pointer(up, es, "up weights")) return q;
  if (rar_result_t q = check_pointer(ids, 8, "ids")) return q;
  reads.push_back(flat(up, adapters * outer * rank * (int64_t)es, "up weights"));
  reads.push_back(flat(ids, tokens * 8, "ids"));
  if (scales) {
    if (rar_result_t q = check_pointer(scales, 4, "scales")) return q;
    reads.push_back(flat(scales, adapters * 4, "scales"));
  }
  const Parts parts = cut_parts(widths, nranks, tokens, dtype);
  const size_t need = (size_t)parts.first[nranks] * tokens * rank * 4;
  if (workspace_bytes < need)
    return set_error(RAR_INVALID_ARGUMENT, "workspace holds " + std::to_string(workspace_bytes) + " bytes, " +
                                               std::to_string(need) + " needed");
  if (need) {
    if (rar_result_t q = check_pointer(workspace, 16, "workspace")) return q;
    writes.push_back(flat(workspace, (int64_t)need, "workspace"));
    scratch.push_back(writes.back());
  }
  if (rar_result_t q = check_blocks(reads, writes, false)) return q;
  if (rar_result_t q = check_blocks(partial_reads, writes, true)) return q;
  if (rar_result_t q = check_blocks(partial_reads, scratch, false)) return q;
  for (int r = 0; r <= nranks; ++r) s.part0[r] = parts.first[r];
  s.ids = e.ids = ids;
  s.h = static_cast<float*>(workspace);
  e.h = s.h;
  s.tokens = e.tokens = tokens;
  s.nranks = e.nranks = nranks;
  s.adapters = e.adapters = (int32_t)adapters;
  s.rank = e.rank = rank;
  s.part_width = parts.width;
  e.up = up;
  e.scales = scales;
  e.ncopies = ncopies;
  e.outer = (int32_t)outer;
  e.parts = parts.first[nranks];
  const int64_t tiles = (tokens + 15) / 16;
  const bool bf = dtype == RAR_BFLOAT16;
  if (e.parts) {
    // Few tiles: a workgroup for every adapter a tile can hold.
    s.slots = tiles <= 16 ? 16 : 1;
    const void* fn = bf ? pick_shrink<BF16>(rank) : pick_shrink<F32>(rank);
    if (rar_result_t q = launch_kernel(fn, dim3((unsigned)tiles, (unsigned)e.parts, (unsigned)s.slots), dim3(kThreads), &s, stream))
      return q;
  }
  const int64_t cols = (outer + 64 * kWaves - 1) / (64 * kWaves);
  e.tiles_per_block = (int32_t)std::max<int64_t>((tiles + 65534) / 65535, std::min<int64_t>(8, tiles * cols / 2048));
  const void* fn = bf ? pick_expand<BF16>(rank) : pick_expand<F32>(rank);
  return launch_kernel(fn, dim3((unsigned)cols, (unsigned)((tiles + e.tiles_per_block - 1) / e.tiles_per_block)), dim3(kThreads), &e,
                       stream);
}

}  // namespace
}  // namespace rar

extern "C" {

rar_result_t rar_adapter_workspace(const int64_t* widths, int nranks, int64_t tokens, rar_dtype_t dtype, int rank,
                                   size_t* bytes) {
  return rar::guarded([&]() -> rar_result_t {
    if (!bytes) return rar::set_error(RAR_INVALID_ARGUMENT, "bytes is NULL");
    if (rar_result_t r = rar::check_adapters(widths, nranks, tokens, dtype, 1, rank)) return r;
    *bytes = (size_t)rar::cut_parts(widths, nranks, tokens, dtype).first[nranks] * tokens * rank * 4;
    return RAR_SUCCESS;
  });
}

rar_result_t rar_adapter_allreduce(const void* const* xs, const int64_t* widths, const int64_t* x_strides,
                                   const void* const* partials, const int64_t* partial_strides, int nranks,
                                   void* const* recvbufs, const int64_t* recv_strides, int nrecv, int64_t tokens,
                                   int64_t outer, rar_dtype_t dtype, const void* const* downs, const void* up,
                                   int64_t adapters, int rank, const int64_t* ids, const float* scales,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  return rar::guarded([&] {
    return rar::adapter_call(xs, widths, x_strides, partials, partial_strides, nranks, recvbufs, recv_strides, nrecv,
                             tokens, outer, dtype, downs, up, adapters, rank, ids, scales, workspace, workspace_bytes,
                             stream);
  });
}

}  // extern "C"
