// paged_decode.cu -- attention of one new token per sequence over its paged cache
// (m.lqnn.cn/news/205170, section "KDA 与 Gated Attention：每 4 层只留 1 层全注意力": the
// softmax-attention layer with its sigmoid output gate).
//
// Per (sequence, query head), over the slots j < len:  s_j = scale q . K_j,  w = softmax(s),
// o = sum_j w_j V_j, o *= sigmoid(z); the weights are added to acc per key-value head.
#include "paged.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float block_reduce(float x, bool is_max, float* buf) {
    for (int o = 16; o > 0; o >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, x, o);
        x = is_max ? fmaxf(x, y) : x + y;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    x = buf[0];
    for (int w = 1; w < kThreads / 32; ++w) x = is_max ? fmaxf(x, buf[w]) : x + buf[w];
    return x;
}

// One CTA per (sequence, query head); w holds [N * Hq, max_len] scores, then weights.
template <typename T>
__global__ void __launch_bounds__(kThreads) decode_kernel(const DecodeArgs a) {
    __shared__ float s_q[128], s_buf[kThreads / 32];
    const int64_t nh = blockIdx.x, n = nh / a.Hq;
    const int hkv = (int)(nh % a.Hq) / (a.Hq / a.H), d = a.d;
    const int len = checked_len(a.seqlens[n], a.max_len, a.c.err);
    float* w = static_cast<float*>(a.workspace) + nh * a.max_len;
    if (threadIdx.x < d) s_q[threadIdx.x] = to_f32(static_cast<const T*>(a.q)[nh * d + threadIdx.x]) * a.scale;
    __syncthreads();
    float m = -INFINITY;
    for (int j = threadIdx.x; j < len; j += kThreads) {
        const int64_t off = slot_offset(a.c, n, j);
        float s = -INFINITY;
        if (off >= 0) {
            const T* k = static_cast<const T*>(a.c.k) + off + hkv * a.c.head_stride;
            s = 0.f;
            for (int c = 0; c < d; ++c) s = fmaf(s_q[c], to_f32(k[c]), s);
        }
        w[j] = s;
        m = fmaxf(m, s);
    }
    m = block_reduce(m, true, s_buf);
    if (m == -INFINITY) m = 0.f;
    float l = 0.f;
    for (int j = threadIdx.x; j < len; j += kThreads) l += (w[j] = expf(w[j] - m));
    l = block_reduce(l, false, s_buf);
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int j = threadIdx.x; j < len; j += kThreads) w[j] *= inv;
    __syncthreads();
    if (threadIdx.x >= d) return;
    float o = 0.f;
    for (int j = 0; j < len; ++j) {
        const int64_t off = slot_offset(a.c, n, j);
        if (off < 0) continue;
        o = fmaf(w[j], to_f32(static_cast<const T*>(a.c.v)[off + hkv * a.c.head_stride + threadIdx.x]), o);
    }
    if (a.z != nullptr) o /= 1.f + expf(-to_f32(static_cast<const T*>(a.z)[nh * d + threadIdx.x]));
    static_cast<T*>(a.o)[nh * d + threadIdx.x] = from_f32<T>(o);
}

// acc[n, h, j] += the sum of the group's weights.
__global__ void __launch_bounds__(kThreads) weights_kernel(const DecodeArgs a) {
    const int64_t nh = blockIdx.x, n = nh / a.H;
    const int h = (int)(nh % a.H), g = a.Hq / a.H;
    const int len = checked_len(a.seqlens[n], a.max_len, a.c.err);
    const float* w = static_cast<const float*>(a.workspace) + (n * a.Hq + h * g) * (int64_t)a.max_len;
    for (int j = threadIdx.x; j < len; j += kThreads) {
        float s = 0.f;
        for (int i = 0; i < g; ++i) s += w[(int64_t)i * a.max_len + j];
        a.acc[nh * a.slots + j] += s;
    }
}

}  // namespace

bool paged_decode_workspace(int64_t N, int64_t Hq, int64_t, int, int64_t max_len, bool, size_t* bytes) {
    const double want = (double)N * Hq * max_len * 4;
    if (want > 9e18) return false;
    *bytes = (size_t)(N * Hq) * (size_t)max_len * 4;
    return true;
}

cudaError_t launch_paged_decode(const DecodeArgs& a, cudaStream_t stream) {
    if (a.N == 0) return cudaSuccess;
    const unsigned grid = (unsigned)(a.N * a.Hq);
    if (a.io == Io::BF16) decode_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(a);
    else decode_kernel<float><<<grid, kThreads, 0, stream>>>(a);
    if (a.acc != nullptr) weights_kernel<<<(unsigned)(a.N * a.H), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
