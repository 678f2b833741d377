// Element types and small helpers shared by the layer operators around the
// scan (gated linear recurrence, add + RMS norm, row quantiser, 8-bit integer
// product).  Activations are fp32, bf16 or fp16; every sum, state, norm and
// statistic is held in fp32 (or in exact integers).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "scan_common.cuh"

namespace ssm {

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

template <class T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T *p)
{
    return *reinterpret_cast<const Vec<T, V> *>(p);
}

template <class T, int V>
__device__ __forceinline__ void store_vec(T *p, const Vec<T, V> &v)
{
    *reinterpret_cast<Vec<T, V> *>(p) = v;
}

__device__ __forceinline__ int ld_acquire(const int *p)
{
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];\n" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void st_release(int *p, int v)
{
    asm volatile("st.release.gpu.global.s32 [%0], %1;\n" ::"l"(p), "r"(v) : "memory");
}

// Debug mode (SSM_SCAN_CHECK=1; api.cu): whether it is on, the sequence table
// checked on the host, and a kernel's status word read back.  The last two
// synchronise and return an ssm_status.
bool debug_checks();
bool debug_fail_waits();                  // SSM_SCAN_TEST_FAIL_WAITS=1: bounded waits give up at once
int debug_check_sequences(const int32_t *seq_starts, const int32_t *seq_lens, int n_seqs, int n_tokens,
                          cudaStream_t stream);
int debug_read_status(const int *status, cudaStream_t stream);

// add_norm.cu.  w null: the row quantiser.  dx, dr: types of x / y and of the residual.
cudaError_t launch_add_norm(const void *x, const void *residual, const float *w, float eps, void *h, void *y,
                            int8_t *codes, float *scales, int rows, int D, int dx, int dr, long long sx,
                            long long sr, long long sh, long long sy, cudaStream_t st);
int add_norm_parts(int rows);             // rows of the gradient's workspace ([parts][D] fp32)
cudaError_t launch_add_norm_backward(const void *gy, const void *h, const void *gh, const float *w, float eps,
                                     void *gin, float *gw, float *part, int rows, int D, int dy, int dr,
                                     long long sgy, long long sh, long long sgh, long long sgi, cudaStream_t st);

// int8_matmul.cu
size_t int8_matmul_workspace_bytes(const void *x, const void *w, int M, int N, int K, long long sx, long long sw);
cudaError_t launch_int8_matmul(const int8_t *x, const float *xs, const int8_t *w, const float *ws, const float *bias,
                               void *out, int M, int N, int K, int dtype, long long sx, long long sw, long long so,
                               void *workspace, cudaStream_t st);

}  // namespace ssm
