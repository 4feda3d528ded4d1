// Accumulated attention weights: after the attention of a step (which leaves log2 of every query
// row's softmax denominator in p.lse), each attended cell gets the sum of its probabilities over
// the query rows of its KV head,
//     w[cell(j)] += sum_r 2^(scale_log2 <q_r, k_j> - lse_r),     rows r = t G + h that see j,
// and the cell of a token appended by this call gets the sum alone. Every key is read from the
// cache (the append has run). One thread owns a cell's sum, so nothing depends on an order; it
// is added with one reduction, so sequences that share a page each add theirs.

struct WeightParams {
    const __nv_bfloat16 *q;          // [B][T][Hq][64]
    const uint8_t *k_cache;          // bf16 pages, or fp8 blocks
    float *weights;                  // [num_pages][Hkv][16]
    const int *block_table, *seq_lens, *q_lens;
    const float *lse;                // [B * Hkv][lse_ld]
    int lse_ld;
    float scale_log2;
    int B, Hq, Hkv, G, T, window, max_pages, num_pages, max_seq_len;
    int assign_new;                  // the call appended its new tokens
};

template <bool KV8>
__global__ void __launch_bounds__(256) weights_plain_kernel(const WeightParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = blockIdx.y, b = blockIdx.z;
    int L = __ldg(p.seq_lens + b);
    int n = p.q_lens != nullptr ? __ldg(p.q_lens + b) : p.T;
    if (L < 0 || L > p.max_seq_len || L > p.max_pages * kPage || n < 0 || n > p.T || n > L) return;
    if (n == 0) return;
    const int base = L - n;
    const int lo0 = p.window > 0 ? max(0, base - p.window + 1) : 0;
    const int tile = lo0 / kPage + blockIdx.x * 8 + warp;
    if (tile * kPage >= L) return;
    const int page = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + tile);
    if (page < 0 || page >= p.num_pages) return;
    const int tok = lane >> 1, d0 = 32 * (lane & 1);
    const int j = tile * kPage + tok;
    float k[32];
    const size_t cell = (static_cast<size_t>(page) * p.Hkv + g) * kPage + tok;
    if constexpr (KV8) {
        const uint8_t *blk = p.k_cache + (static_cast<size_t>(page) * p.Hkv + g) * kBlk8Bytes;
        const float sc = reinterpret_cast<const float *>(blk + kBlk8S)[tok];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t lo, hi;
            e4m3x4_to_f16x2x2(*reinterpret_cast<const uint32_t *>(blk + tok * kD + d0 + 4 * i), lo, hi);
            const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&lo)), c = __half22float2(*reinterpret_cast<__half2 *>(&hi));
            k[4 * i] = a.x * sc;
            k[4 * i + 1] = a.y * sc;
            k[4 * i + 2] = c.x * sc;
            k[4 * i + 3] = c.y * sc;
        }
    } else {
        const uint32_t *row = reinterpret_cast<const uint32_t *>(p.k_cache + cell * kD * 2) + d0 / 2;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 a = unpack_bf16(row[i]);
            k[2 * i] = a.x;
            k[2 * i + 1] = a.y;
        }
    }
    float sum = 0.f;
    const float *lse = p.lse + (static_cast<size_t>(b) * p.Hkv + g) * p.lse_ld;
    for (int t = 0; t < n; ++t)
        for (int h = 0; h < p.G; ++h) {
            const uint32_t *qr = reinterpret_cast<const uint32_t *>(
                p.q + ((static_cast<size_t>(b) * p.T + t) * p.Hq + g * p.G + h) * kD + d0);
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 a = unpack_bf16(__ldg(qr + i));
                dot += a.x * k[2 * i] + a.y * k[2 * i + 1];
            }
            dot += __shfl_xor_sync(0xffffffffu, dot, 1);
            const bool see = j <= base + t && (p.window == 0 || j > base + t - p.window);
            if (see) sum += fast_exp2(dot * p.scale_log2 - __ldg(lse + t * p.G + h));
        }
    if ((lane & 1) == 0 && j < L && j >= lo0) {
        if (p.assign_new && j >= base)
            p.weights[cell] = sum;
        else
            atomicAdd(p.weights + cell, sum);
    }
}
