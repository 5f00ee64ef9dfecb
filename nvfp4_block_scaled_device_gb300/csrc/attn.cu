// Causal attention with grouped heads, over packed prompts or the paged cache:
//   s_j = scale * q.k_j over the keys j a row sees, out = sum_j softmax_j(s) v_j.
//
// One warp per (packed row, head); lane l holds columns 4l .. 4l+3.  The keys
// are taken one after the other with the running maximum m and sum l of the
// softmax: m' = max(m, s), l' = l e^(m-m') + e^(s-m'), o' = o e^(m-m') +
// e^(s-m') v.
#include "attn.h"
#include "common.cuh"
#include "internal.h"

namespace nvfp4 {
namespace {

constexpr int kWarps = 4;

struct Params {
    nvfp4_step_t s;
    nvfp4_attn_io_t io;
    AttnKV kv;
};

__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* f)
{
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    f[0] = bf16_lo(w.x);
    f[1] = bf16_hi(w.x);
    f[2] = bf16_lo(w.y);
    f[3] = bf16_hi(w.y);
}

__global__ void __launch_bounds__(kWarps * 32) attn_row_kernel(const Params p)
{
    const int H = (int)p.s.heads, D = (int)p.io.head_dim;
    const int group = H / (int)p.s.kv_heads;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t row = w / H;
    const int h = (int)(w % H), hk = h / group;
    if (row >= p.s.cu_q[p.s.requests]) return;
    int lo = 0, hi = (int)p.s.requests - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.s.cu_q[mid] <= row) lo = mid; else hi = mid - 1;
    }
    const int64_t first = p.s.cu_q[lo], q_len = p.s.cu_q[lo + 1] - first, kv_len = p.s.kv_len[lo];
    const int64_t pos = kv_len - q_len + (row - first);
    const bool on = 4 * lane < D;
    const bool paged = p.kv.block_table != nullptr;
    float q[4] = {0.f, 0.f, 0.f, 0.f}, o[4] = {0.f, 0.f, 0.f, 0.f}, k[4], v[4];
    if (on) load4(static_cast<const __nv_bfloat16*>(p.io.q) + row * p.io.ldq + h * p.io.hq + 4 * lane, q);
    float m = -INFINITY, l = 0.f;
    int64_t j0 = p.s.window && pos + 1 > p.s.window ? pos + 1 - p.s.window : 0, j1 = pos + 1;
    if (paged && j1 > p.kv.table_cols * p.kv.page_size) j1 = p.kv.table_cols * p.kv.page_size;
    for (int64_t j = j0; j < j1; j++) {
        const __nv_bfloat16 *pk, *pv;
        bool real = true;
        if (paged) {
            const int64_t page = p.kv.block_table[lo * p.kv.table_ld + j / p.kv.page_size];
            real = page >= 0 && page < p.kv.pages;
            const int64_t at =
                (real ? page : 0) * p.kv.page_stride + (hk * p.kv.page_size + j % p.kv.page_size) * D + 4 * lane;
            pk = p.kv.k + at;
            pv = p.kv.v + at;
        } else {
            pk = p.kv.k + (first + j) * p.kv.ldk + hk * p.kv.hk + 4 * lane;
            pv = p.kv.v + (first + j) * p.kv.ldv + hk * p.kv.hv + 4 * lane;
        }
        float s = 0.f;
        if (on && real) {
            load4(pk, k);
            load4(pv, v);
#pragma unroll
            for (int i = 0; i < 4; i++) s += q[i] * k[i];
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) v[i] = 0.f;
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= p.io.scale;
        const float m1 = fmaxf(m, s);
        const float ms = m1 == -INFINITY ? 0.f : m1;
        const float a = expf(m - ms), e = expf(s - ms);
        l = l * a + e;
#pragma unroll
        for (int i = 0; i < 4; i++) o[i] = o[i] * a + e * v[i];
        m = m1;
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    if (on) {
        uint2 w2;
        w2.x = cvt_bf16x2(o[0] * inv, o[1] * inv);
        w2.y = cvt_bf16x2(o[2] * inv, o[3] * inv);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.io.out) + row * p.io.ldo + h * p.io.ho + 4 * lane) = w2;
    }
    if (p.io.lse && lane == 0) p.io.lse[row * H + h] = l > 0.f || l != l ? m + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t launch_attn(const nvfp4_step_t& step, const nvfp4_attn_io_t& io, const AttnKV& kv, int num_sms,
                        cudaStream_t stream)
{
    (void)num_sms;
    const Params p = {step, io, kv};
    const int64_t warps = step.tokens * step.heads;
    attn_row_kernel<<<(unsigned)((warps + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace nvfp4
