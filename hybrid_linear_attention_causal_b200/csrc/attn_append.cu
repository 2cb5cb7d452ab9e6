// Quantises new key and value rows into the paged 8-bit cache.
//
// One block per (request, page it touches, key/value head, keys or values).  The block reads its new rows
// once into registers, takes the largest magnitude, settles the page's exponent (the smallest e with
// amax <= 448 * 2^e, not below that of tokens already in the page), multiplies by 2^-e (exact) and rounds
// to e4m3.  A page whose exponent rises has its earlier codes multiplied by the power of two between the
// exponents and rounded again, which changes only codes that become subnormal.  The work is a copy: bytes
// should bound it for a prefill batch, the launch and a few dependent reads do for a decode step.  Measured (B200):
// 22860 rows of 8 heads of 128, 140 MB: 33 us, 4.2 TB/s (instructions: eight or so a value); 64 rows: 5.3 us.

#include "attn_internal.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace attn {
namespace {

// the smallest e in ATTN_EXP_MIN .. ATTN_EXP_MAX with amax <= 448 * 2^e (448 = 1.75 * 2^8)
__device__ __forceinline__ int block_exponent(float amax) {
    const int bits = __float_as_int(amax);
    const int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
    return max(ATTN_EXP_MIN, min(ATTN_EXP_MAX, e));  // zero and subnormal amax fall below the range
}

// two floats -> two e4m3 codes (nearest even, saturating), the first in the low byte
__device__ __forceinline__ uint32_t narrow2(float x0, float x1) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(x0), "f"(x1));
    return r;
}

// Block (i, 2 h + keys or values).  With cu_seqlens, request n owns blocks f(n) .. f(n+1)-1, where
// f(n) = cu[n] / ps + 2 n: at least as many as the pages that its rows can touch, without a scan.
// NV: 16-byte vectors per thread that hold a page of rows.
template <typename T, int D, int NV, int NT>
__global__ void __launch_bounds__(NT) append_kernel(const __grid_constant__ AppendArgs p) {
    constexpr int kN = Vec16<T>::kN, kPerRow = D / kN;  // vectors of a row
    __shared__ int s_n, s_row0, s_len, s_start;
    __shared__ float s_max[NT / 32];
    __shared__ int s_bad;
    const int tid = threadIdx.x, ps = 1 << p.ps_shift;
    const int kv = blockIdx.y & 1, h = blockIdx.y >> 1;
    int n, idx, row0, L, start;
    if (p.cu) {
        if (tid == 0) s_n = -1, s_bad = 0;
        __syncthreads();
        bool bad = tid == 0 && p.cu[0] != 0;
        for (int i = tid; i < p.N; i += NT) {
            const int c0 = p.cu[i], c1 = p.cu[i + 1];
            if (c0 < 0 || c1 < c0 || c1 > p.T) {
                bad = true;
                continue;
            }
            const int f0 = (c0 >> p.ps_shift) + 2 * i, f1 = (c1 >> p.ps_shift) + 2 * i + 2;
            if (f0 <= (int)blockIdx.x && (int)blockIdx.x < f1) s_n = i, s_row0 = c0, s_len = c1 - c0, s_start = p.start[i];
        }
        if (bad) s_bad = 1;
        __syncthreads();
        if (s_bad) {
            if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) raise_error(p.hdr, GDN_DEVERR_SEQLENS);
            return;
        }
        n = s_n;
        if (n < 0) return;
        row0 = s_row0;
        L = s_len;
        start = s_start;
        idx = (int)blockIdx.x - (row0 >> p.ps_shift) - 2 * n;
    } else {
        const int per_req = ((p.per + ps - 2) >> p.ps_shift) + 1;
        n = blockIdx.x / per_req;
        idx = blockIdx.x - n * per_req;
        row0 = n * p.per;
        L = p.per;
        start = p.start[n];
    }
    if (start < 0 || L == 0) return;  // padding
    if ((long long)start + L > ((long long)p.max_pages << p.ps_shift)) {
        if (tid == 0) raise_error(p.hdr, GDN_DEVERR_KV_LEN);
        return;
    }
    const int pi = (start >> p.ps_shift) + idx;     // page of the request
    const int t0 = max(start, pi << p.ps_shift);    // tokens [t0, t1) of the request go into it
    const int t1 = min(start + L, (pi + 1) << p.ps_shift);
    if (t0 >= t1) return;
    const int r0 = t0 & (ps - 1), count = t1 - t0;
    const T* src = static_cast<const T*>(p.x[kv]) + (long long)(row0 + t0 - start) * p.stride[kv] + (long long)h * D;

    uint4 w[NV];  // on their way while the page is looked up
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = i * NT + tid, r = e / kPerRow;
        if (r < count) w[i] = *reinterpret_cast<const uint4*>(src + (long long)r * p.stride[kv] + (e % kPerRow) * kN);
    }
    const int page = p.table[(long long)n * p.max_pages + pi];
    if (page < 0 || page >= p.num_pages) {
        if (tid == 0) raise_error(p.hdr, GDN_DEVERR_PAGE_RANGE);
        return;
    }
    const long long block = (long long)page * p.HKV + h;
    uint8_t* dst = p.codes[kv] + (block << p.ps_shift) * D;
    int8_t* exp_at = p.exps[kv] + block;

    const int e_old = r0 > 0 ? *exp_at : ATTN_EXP_MIN;
    float amax = 0.0f;
    bool odd = false;  // an inf or a NaN: it takes no part in the exponent
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if ((i * NT + tid) / kPerRow < count) {
            float x[kN];
            Vec16<T>::get(w[i], x);
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                const float a = fabsf(x[j]);
                if (a < INFINITY) amax = fmaxf(amax, a);
                else odd = true;
            }
        }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((tid & 31) == 0) s_max[tid >> 5] = amax;
    odd = __syncthreads_or(odd) != 0;  // every thread has read the old exponent before one writes the new
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) amax = fmaxf(amax, s_max[i]);
    if (odd && tid == 0) raise_error(p.hdr, GDN_DEVERR_NONFINITE);
    const int e_new = max(e_old, block_exponent(amax));
    if (tid == 0) *exp_at = (int8_t)e_new;

    const float f = __int_as_float((127 - e_new) << 23);  // 2^-e_new
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = i * NT + tid, r = e / kPerRow;
        if (r < count) {
            float x[kN];
            Vec16<T>::get(w[i], x);
#pragma unroll
            for (int j = 0; j < kN; ++j) x[j] = isnan(x[j]) ? 0.0f : x[j] * f;
            uint8_t* at = dst + (r0 + r) * D + (e % kPerRow) * kN;
            const uint32_t c0 = narrow2(x[0], x[1]) | narrow2(x[2], x[3]) << 16;
            if constexpr (kN == 8) {
                const uint32_t c1 = narrow2(x[4], x[5]) | narrow2(x[6], x[7]) << 16;
                *reinterpret_cast<uint2*>(at) = make_uint2(c0, c1);
            } else {
                *reinterpret_cast<uint32_t*>(at) = c0;
            }
        }
    }
    if (r0 > 0 && e_new > e_old) {
        const float g = ldexpf(1.0f, e_old - e_new);
        for (int e = tid; e < r0 * (D / 4); e += NT) {
            const uint32_t c = reinterpret_cast<uint32_t*>(dst)[e];
            float x[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t hh;
                const uint16_t two = (uint16_t)(c >> (16 * i));
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hh) : "h"(two));
                const float2 y = tc::unpack_f16(hh);
                x[2 * i] = y.x * g, x[2 * i + 1] = y.y * g;
            }
            reinterpret_cast<uint32_t*>(dst)[e] = narrow2(x[0], x[1]) | narrow2(x[2], x[3]) << 16;
        }
    }
}

template <typename T, int D>
cudaError_t launch_dim(const AppendArgs& p, cudaStream_t s) {
    const int ps = 1 << p.ps_shift;
    const long long blocks = p.cu ? (long long)(p.T >> p.ps_shift) + 2LL * p.N
                                  : (long long)p.N * (((p.per + ps - 2) >> p.ps_shift) + 1);
    const dim3 grid((unsigned)blocks, 2 * p.HKV);
    // a page of rows is 2 to 64 KB: at most 16 vectors of it per thread
    const int rows = p.cu || p.per > ps ? ps : p.per;
    const long long bytes = (long long)rows * D * sizeof(T);
    if (bytes <= 2048) append_kernel<T, D, 1, 128><<<grid, 128, 0, s>>>(p);
    else if (bytes <= 8192) append_kernel<T, D, 4, 128><<<grid, 128, 0, s>>>(p);
    else if (bytes <= 16384) append_kernel<T, D, 8, 128><<<grid, 128, 0, s>>>(p);
    else append_kernel<T, D, 16, 256><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const AppendArgs& p, int D, int dtype, cudaStream_t s) {
    if (dtype == GDN_DTYPE_F32) return D == 128 ? launch_dim<float, 128>(p, s) : launch_dim<float, 64>(p, s);
    return D == 128 ? launch_dim<__nv_bfloat16, 128>(p, s) : launch_dim<__nv_bfloat16, 64>(p, s);
}

}  // namespace attn
}  // namespace gdn
