// 8-bit integer matrix product with a scale for each token and each output
// channel (sm_103a):
//
//   out[t][n] = (sum_k xq[t][k] wq[n][k]) xs[t] ws[n] + bias[n]
//
// The sum is an exact integer (inner <= 131071 keeps it inside 32 bits).
#include "layer_common.cuh"

namespace ssm {

namespace {

struct I8Args {
    const int8_t *x, *w;
    const float *xs, *ws, *bias;
    void *out;
    int M, N, K;
    long long sx, sw, so;
};

constexpr int kTile = 64, kStep = 64;

// 64 x 64 outputs a block, 4 x 4 a thread, packed 4-term integer products.
template <class T>
__global__ void __launch_bounds__(256)
int8_matmul_kernel(const I8Args a)
{
    griddep_entry();
    __shared__ int xt[kTile][kStep / 4 + 1], wt[kTile][kStep / 4 + 1];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const long long m0 = (long long)blockIdx.x * kTile, n0 = (long long)blockIdx.y * kTile;
    int acc[4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += kStep) {
        for (int i = tid; i < kTile * kStep / 4; i += 256) {
            const int r = i / (kStep / 4), c = i % (kStep / 4);
            unsigned xv = 0, wv = 0;
            for (int b = 0; b < 4; ++b) {
                const int k = k0 + 4 * c + b;
                if (k < a.K) {
                    if (m0 + r < a.M)
                        xv |= (unsigned)(uint8_t)a.x[(m0 + r) * a.sx + k] << (8 * b);
                    if (n0 + r < a.N)
                        wv |= (unsigned)(uint8_t)a.w[(n0 + r) * a.sw + k] << (8 * b);
                }
            }
            xt[r][c] = (int)xv;
            wt[r][c] = (int)wv;
        }
        __syncthreads();
        for (int c = 0; c < kStep / 4; ++c) {
            int xv[4], wv[4];
            for (int i = 0; i < 4; ++i) {
                xv[i] = xt[ty + 16 * i][c];
                wv[i] = wt[tx + 16 * i][c];
            }
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __dp4a(xv[i], wv[j], acc[i][j]);
        }
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const long long m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m < a.M && n < a.N) {
                float v = (float)acc[i][j] * a.xs[m] * a.ws[n];
                if (a.bias)
                    v += a.bias[n];
                static_cast<T *>(a.out)[m * a.so + n] = from_float<T>(v);
            }
        }
}

}  // namespace

size_t int8_matmul_workspace_bytes(int, int, int) { return 0; }

cudaError_t launch_int8_matmul(const int8_t *x, const float *xs, const int8_t *w, const float *ws, const float *bias,
                               void *out, int M, int N, int K, int dtype, long long sx, long long sw, long long so,
                               void *, cudaStream_t st)
{
    const I8Args a{x, w, xs, ws, bias, out, M, N, K, sx, sw, so};
    const dim3 grid((unsigned)((M + kTile - 1) / kTile), (unsigned)((N + kTile - 1) / kTile));
    switch (dtype) {
    case kF32: return launch_pdl(int8_matmul_kernel<float>, grid, dim3(256), 0, st, a);
    case kBF16: return launch_pdl(int8_matmul_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, a);
    case kF16: return launch_pdl(int8_matmul_kernel<__half>, grid, dim3(256), 0, st, a);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace ssm
