// gdp_block.cuh -- what the operators of gdp_block.h share: packed sequences, state modes, vectors of channels,
// and the host's checks.
#pragma once

#include <climits>
#include <initializer_list>

#include "../../include/gdp_block.h"
#include "gdp_layer.cuh"
#include "gdp_sm100.cuh"

namespace gdp {
namespace layer {

int sm_count();  // of the current device (gdp_recurrence.cu)

// ---- packed sequences ----
struct Packed {
  const void *cu;
  int cu64;
  int64_t T, N;
  uint32_t *status;
};
__device__ __forceinline__ int64_t cu_at(const Packed &p, int64_t i) {
  const int64_t v = p.cu64 ? static_cast<const int64_t *>(p.cu)[i] : (int64_t) static_cast<const int32_t *>(p.cu)[i];
  return max((int64_t)0, min(v, p.T));
}
// Rows [b, e) of sequence i, within the tensors whatever cu_seqlens holds.
__device__ __forceinline__ void seq_rows(const Packed &p, int64_t i, int64_t *b, int64_t *e) {
  *b = cu_at(p, i);
  *e = max(*b, cu_at(p, i + 1));
}
// The last sequence that begins at or before row t (the one that holds t, where t is no padding).
__device__ __forceinline__ int64_t seq_of_row(const Packed &p, int64_t t) {
  int64_t lo = 0, hi = p.N - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if (cu_at(p, mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
// One CTA's threads: the status bit of bounds that do not ascend from 0 to at most T.
__device__ __forceinline__ void check_packed(const Packed &p) {
  bool bad = false;
  for (int64_t i = threadIdx.x + (int64_t)threadIdx.y * blockDim.x; i <= p.N; i += blockDim.x * blockDim.y) {
    const int64_t v = p.cu64 ? static_cast<const int64_t *>(p.cu)[i] : (int64_t) static_cast<const int32_t *>(p.cu)[i];
    bad |= v < 0 || v > p.T || (i == 0 && v != 0) || (i > 0 && cu_at(p, i - 1) > v);
  }
  if (bad) set_status(p.status, GDP_DEV_ERR_CU_SEQLENS);
}

// ---- state modes ----
struct StateModes {
  const void *init;
  void *fin, *cache;
  const int32_t *slots;
  int64_t num_slots;
};
// Index of sequence i's state in the cache, -1 for none.
__device__ __forceinline__ int64_t slot_of(const StateModes &s, int64_t i, uint32_t *status, bool report) {
  const int64_t slot = s.slots[i];
  if (slot >= 0 && slot < s.num_slots) return slot;
  if (slot != -1 && report) set_status(status, GDP_DEV_ERR_SLOT);
  return -1;
}
// Where sequence i's state of `elems` elements is read (NULL: zero) and written (NULL: nowhere).
template <typename T>
__device__ __forceinline__ void state_of(const StateModes &s, int64_t i, int64_t elems, uint32_t *status, bool report, const T **src, T **dst) {
  if (s.cache) {
    const int64_t slot = slot_of(s, i, status, report);
    *dst = slot >= 0 ? static_cast<T *>(s.cache) + slot * elems : nullptr;
    *src = *dst;
  } else {
    *src = s.init ? static_cast<const T *>(s.init) + i * elems : nullptr;
    *dst = s.fin ? static_cast<T *>(s.fin) + i * elems : nullptr;
  }
}

// ---- vectors of channels ----
template <typename T, int V>
struct alignas(V * sizeof(T)) Vec {
  T v[V];
};
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T *at) { return *reinterpret_cast<const Vec<T, V> *>(at); }
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *at, const float *v) {
  Vec<T, V> o;
#pragma unroll
  for (int k = 0; k < V; ++k) o.v[k] = from_f32<T>(v[k]);
  *reinterpret_cast<Vec<T, V> *>(at) = o;
}

// sigmoid(v) with the hardware's exponential and reciprocal (relative error about 2^-21 + |v| 2^-24; below
// -87.3 it is 0, as e^-v leaves fp32).
__device__ __forceinline__ float sigmoid_fast(float v) { return rcp(1.f + exp_fast(-v)); }

__device__ __forceinline__ float2 sigmoid2(float2 v) {
  const float2 t = mul2(v, both(-kLog2e)), d = add2(make_float2(ex2(t.x), ex2(t.y)), both(1.f));
  return make_float2(rcp(d.x), rcp(d.y));
}

// ---- host side ----
// A [T, C] tensor: given where it has elements, aligned to its elements, rows at least C apart.
inline gdp_status rows_ok(const void *p, int64_t stride, int64_t T, int64_t C, int type, const char *name) {
  if (T > 0 && !p) {
    set_last_error("%s is required", name);
    return GDP_ERR_INVALID_ARG;
  }
  if (!aligned(p, dtype_size(type)) || (T > 1 && stride < C)) {
    set_last_error("%s must be aligned to its elements, its rows at least C elements apart", name);
    return GDP_ERR_INVALID_ARG;
  }
  return GDP_OK;
}
// The stride of a single row means nothing and may be anything in a view.
inline int64_t stride_of(int64_t stride, int64_t T, int64_t C) { return T > 1 ? stride : C; }
// A tensor of T rows as the overlap checks see it: `cols` elements every `stride` (an output's are contiguous), in `groups`
// that are `stride_g` apart.
struct Span {
  const void *p;
  int64_t stride, cols;
  int type;
  const char *name;
  int64_t groups, stride_g;
};
inline Span rows(const void *p, int64_t stride, int64_t cols, int type, const char *name) { return {p, stride, cols, type, name, 1, 0}; }
inline Span dense(const void *p, int64_t cols, int type, const char *name) { return rows(p, cols, cols, type, name); }
// Whether T >= 1 rows share memory with T contiguous ones (the gaps between a strided tensor's rows are not its own).
inline bool spans_overlap(const Span &in, const Span &out, int64_t T) {
  if (!in.p || !out.p) return false;
  typedef __int128 Wide;  // (strides may be anything)
  const Wide es = dtype_size(in.type), row = in.cols * es, apart = in.stride * es, bytes = (Wide)T * out.cols * dtype_size(out.type);
  const Wide whole = (T - 1) * apart + (in.groups - 1) * in.stride_g * es + row, d = (Wide)(uintptr_t)out.p - (Wide)(uintptr_t)in.p;
  if (d >= whole || d + bytes <= 0) return false;
  for (int64_t g = 0; g < in.groups; ++g) {
    const Wide at = d - g * in.stride_g * es;  // of the output, from the group's first row
    const Wide t = at < row ? 0 : (at - row) / apart + 1;  // the first row that ends behind the output's begin
    if (t < T && t * apart < at + bytes) return true;
  }
  return false;
}
// Outputs share memory with no input and not with one another.
inline gdp_status apart_ok(int64_t T, std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  if (T == 0) return GDP_OK;
  const Span *o = outs.begin();
  for (size_t i = 0; i < outs.size(); ++i) {
    for (const Span &in : ins)
      if (spans_overlap(in, o[i], T)) {
        set_last_error("%s overlaps %s", o[i].name, in.name);
        return GDP_ERR_ALIAS;
      }
    for (size_t k = 0; k < i; ++k)
      if (spans_overlap(o[k], o[i], T)) {
        set_last_error("%s overlaps %s", o[i].name, o[k].name);
        return GDP_ERR_ALIAS;
      }
  }
  return GDP_OK;
}
// Whether its rows can be read `bytes` at a time.
inline bool rows_by(const void *p, int64_t stride, int64_t T, int type, size_t bytes) {
  return aligned(p, bytes) && (T <= 1 || stride * dtype_size(type) % bytes == 0);
}
inline gdp_status states_ok(const void *init, const void *fin, const void *cache, const int32_t *slots, int64_t num_slots, size_t align,
                            size_t bytes) {
  if (!aligned(init, align) || !aligned(fin, align) || !aligned(cache, align) || !aligned(slots, 4))
    return fail(GDP_ERR_INVALID_ARG, "state buffers must be aligned to their elements");
  if (cache && (init || fin)) return fail(GDP_ERR_INVALID_ARG, "the state cache excludes initial_state and output_state");
  if (cache && (!slots || num_slots < 1)) return fail(GDP_ERR_INVALID_ARG, "the state cache needs state_indices and num_slots >= 1");
  if (partly_overlap(init, fin, bytes)) return fail(GDP_ERR_ALIAS, "output_state partly overlaps initial_state");
  return GDP_OK;
}
inline gdp_status shape_ok(int64_t T, int64_t N, int64_t C) {
  if (T < 0 || N < 0 || C < 1) return fail(GDP_ERR_INVALID_ARG, "T >= 0, N >= 0 and C >= 1 are required");
  if (T > INT32_MAX || N > INT32_MAX - 1 || C > (1 << 20)) return fail(GDP_ERR_UNSUPPORTED, "T below 2^31, N below 2^31 - 1, C up to 2^20");
  return GDP_OK;
}
inline gdp_status cuda_status(cudaError_t e, const char *what) {
  if (e == cudaSuccess) return GDP_OK;
  set_last_error("%s: %s", what, cudaGetErrorString(e));
  return GDP_ERR_CUDA;
}
// Zeros into an output none of whose rows belongs to a sequence.
inline gdp_status zero_out(void *p, size_t elems, int type, cudaStream_t stream) {
  if (!p || elems == 0) return GDP_OK;
  return cuda_status(cudaMemsetAsync(p, 0, elems * dtype_size(type), stream), "padding rows");
}

// Column sums of a workspace [parts][cols] in a fixed order, into out (gdp_conv.cu).
struct ColumnSums {
  const float *from;   // [parts][cols]
  int64_t parts, cols;
  float *to[4];        // column i of segment k goes to to[k][i - first]; NULL: dropped
  int64_t first[4];    // segments' first columns, ascending
  int64_t taps, width; // segment 0 is [taps][width] and goes out transposed, [width][taps] (taps 0: as it is)
};
cudaError_t launch_column_sums(const ColumnSums &s, cudaStream_t stream);

}  // namespace layer
}  // namespace gdp
