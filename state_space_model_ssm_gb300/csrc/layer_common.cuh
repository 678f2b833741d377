// Element types and small helpers shared by the layer operators around the
// scan (gated linear recurrence, add + RMS norm, row quantiser, 8-bit integer
// product).  Activations are fp32, bf16 or fp16; every sum, state, norm and
// statistic is held in fp32 (or in exact integers).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "scan_common.cuh"

namespace ssm {

// SMs of a GB300, the one device this is built for.  Launch shapes count on it; results do not.
constexpr int kSms = 152;

// Element types of the ABI (ssm_dtype).
enum { kF32 = 0, kBF16 = 1, kF16 = 2 };

__host__ __device__ constexpr int dtype_size(int dtype) { return dtype == kF32 ? 4 : 2; }

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

template <class T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// V consecutive elements, loaded and stored as one access of V * sizeof(T)
// bytes (at most 16; the address must be a multiple of that).
template <class T, int V>
struct alignas(sizeof(T) * V) Vec {
    T v[V];
};

// They move as integer words: an access chosen at run time between a vector and its
// elements then has two different types and cannot be merged into one with the
// vector's alignment.
template <int BYTES>
struct WordsOf;
template <>
struct WordsOf<16> { using type = uint4; };
template <>
struct WordsOf<8> { using type = uint2; };
template <>
struct WordsOf<4> { using type = uint32_t; };

template <class T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T *p)
{
    using W = typename WordsOf<sizeof(T) * V>::type;
    Vec<T, V> v;
    *reinterpret_cast<W *>(&v) = *reinterpret_cast<const W *>(p);
    return v;
}

template <class T, int V>
__device__ __forceinline__ void store_vec(T *p, const Vec<T, V> &v)
{
    using W = typename WordsOf<sizeof(T) * V>::type;
    *reinterpret_cast<W *>(p) = *reinterpret_cast<const W *>(&v);
}

// cuTensorMapEncodeTiled, or null without a driver that has it (gated_scan.cu).
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Debug mode (SSM_SCAN_CHECK=1; api.cu): whether it is on, the sequence table
// checked on the host, and a kernel's status word read back.  The last two
// synchronise and return an ssm_status.
bool debug_checks();
// SSM_SCAN_TEST_FAIL_WAITS: 0, 1 (bounded waits give up at once) or 2 (in the gated scan's
// clusters one warp's wait does, from the second round on; else as 1)
int debug_fail_waits();
int debug_check_sequences(const int32_t *seq_starts, const int32_t *seq_lens, int n_seqs, int n_tokens,
                          cudaStream_t stream);

// add_norm.cu.  w null: the row quantiser.  dx, dr: types of x / y and of the residual.
cudaError_t launch_add_norm(const void *x, const void *residual, const float *w, float eps, void *h, void *y,
                            int8_t *codes, float *scales, int rows, int D, int dx, int dr, long long sx,
                            long long sr, long long sh, long long sy, cudaStream_t st);
int add_norm_parts(int rows, int D);      // rows of the gradient's workspace ([parts][D] fp32)
cudaError_t launch_add_norm_backward(const void *gy, const void *h, const void *gh, const float *w, float eps,
                                     void *gin, float *gw, float *part, int rows, int D, int dy, int dr,
                                     long long sgy, long long sh, long long sgh, long long sgi, cudaStream_t st);

// int8_matmul.cu
size_t int8_matmul_workspace_bytes(const void *x, const void *w, int M, int N, int K, long long sx, long long sw);
cudaError_t launch_int8_matmul(const int8_t *x, const float *xs, const int8_t *w, const float *ws, const float *bias,
                               void *out, int M, int N, int K, int dtype, long long sx, long long sw, long long so,
                               void *workspace, cudaStream_t st);

}  // namespace ssm
