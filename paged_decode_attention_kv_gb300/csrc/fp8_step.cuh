// What stands around the attention over an fp8 cache in a step of new tokens: the norms and the
// rotation of the projected queries and keys (qk_norm_rope_kernel), the tokens quantised into
// their blocks (kv_append_fp8_kernel), and cached positions read back as bf16
// (kv_read_fp8_kernel).
//
// Included into decode_attn.cu (inside its anonymous namespace): one translation unit, sharing
// the fp8 helpers and the status word.

// 32 bytes to global memory at a 32-byte aligned address.
__device__ __forceinline__ void st_global_v8(void *p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// ------------------------------------------------------------------ norms and rotation
// Row x of 64 values of one head: y = x w / sqrt(sum(x^2) / 64 + eps) (no norm: y = x), then the
// pairs (i, i + 32) rotated by row pos[axis(i)] of the tables. All in fp32, rounded once to bf16;
// the rotation's products and its sum or difference are rounded one by one, as in the other
// calls with a rotary embedding (without a norm the bits are theirs).
//
// Bound by memory: every row is read and written once. Four lanes hold a row, lane j its
// elements 8 j .. + 7 and 32 + 8 j .. + 7, so that a lane has both halves of its pairs (two
// 16-byte loads and stores, no exchange for the rotation; two shuffles for the norm). A lane
// keeps its pairs' cosines and sines over all the rows of a token that its warp takes.
struct RotateParams {
    const __nv_bfloat16 *q, *k, *v;          // token strides below, heads contiguous; v may be null
    __nv_bfloat16 *q_out, *k_out, *v_out;
    long long q_ld, k_ld, v_ld, qo_ld, ko_ld, vo_ld;  // elements from one token to the next
    const int32_t *positions;                // [axes][N]
    const float *rope_cos, *rope_sin;        // [max_position][32]
    const float *q_weight, *k_weight;        // [64] or null
    float eps;
    int N, Hq, Hkv, max_position;
    int rows, chunk;                         // rows of a token (q, k, v), rows a warp takes of it at most
    unsigned char axis[kD / 2];              // the axis of each pair
    unsigned char quads;                     // bit i: the pairs 4 i .. 4 i + 3 are of one axis
};
constexpr int kRotThreads = 128;
constexpr int kRotRows = 16;

__global__ void __launch_bounds__(kRotThreads) qk_norm_rope_kernel(const __grid_constant__ RotateParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunks = (p.rows + p.chunk - 1) / p.chunk;
    const long long item = static_cast<long long>(blockIdx.x) * (kRotThreads / 32) + warp;
    const long long tok = item / chunks;
    if (tok >= p.N) return;
    const int r_begin = static_cast<int>(item - tok * chunks) * p.chunk, r_end = min(r_begin + p.chunk, p.rows);
    const int j = lane & 3;
    float c[8], s[8];
    if (r_begin < p.Hq + p.Hkv) {
        bool bad = false;
        auto row_of = [&](int a) {
            const int pos = __ldg(p.positions + static_cast<long long>(a) * p.N + tok);
            const bool out = pos < 0 || pos >= p.max_position;
            bad = bad || out;
            return static_cast<size_t>(out ? 0 : pos) * (kD / 2);
        };
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i0 = 8 * j + 4 * h;
            if (p.quads >> (i0 >> 2) & 1) {
                const size_t at = row_of(p.axis[i0]) + i0;
                const float4 cv = __ldg(reinterpret_cast<const float4 *>(p.rope_cos + at));
                const float4 sv = __ldg(reinterpret_cast<const float4 *>(p.rope_sin + at));
                c[4 * h] = cv.x, c[4 * h + 1] = cv.y, c[4 * h + 2] = cv.z, c[4 * h + 3] = cv.w;
                s[4 * h] = sv.x, s[4 * h + 1] = sv.y, s[4 * h + 2] = sv.z, s[4 * h + 3] = sv.w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const size_t at = row_of(p.axis[i0 + e]) + i0 + e;
                    c[4 * h + e] = __ldg(p.rope_cos + at);
                    s[4 * h + e] = __ldg(p.rope_sin + at);
                }
            }
        }
        if (bad) flag_status(DA_STATUS_BAD_POSITION);
    }
    for (int r = r_begin + (lane >> 2); r - (lane >> 2) < r_end; r += 8) {  // (all lanes stay for the shuffles)
        const bool live = r < r_end;
        const int kind = r < p.Hq ? 0 : r < p.Hq + p.Hkv ? 1 : 2;  // q, k, v
        const int h = kind == 0 ? r : kind == 1 ? r - p.Hq : r - p.Hq - p.Hkv;
        const __nv_bfloat16 *src = (kind == 0 ? p.q + tok * p.q_ld : kind == 1 ? p.k + tok * p.k_ld : p.v + tok * p.v_ld) + h * kD + 8 * j;
        __nv_bfloat16 *dst = (kind == 0 ? p.q_out + tok * p.qo_ld : kind == 1 ? p.k_out + tok * p.ko_ld : p.v_out + tok * p.vo_ld) + h * kD + 8 * j;
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (live) {
            a = *reinterpret_cast<const uint4 *>(src);
            b = *reinterpret_cast<const uint4 *>(src + kD / 2);
        }
        const float *w = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
        uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
        float x[8], y[8], ss = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 u = unpack_bf16(aw[e]), v = unpack_bf16(bw[e]);
            x[2 * e] = u.x, x[2 * e + 1] = u.y, y[2 * e] = v.x, y[2 * e + 1] = v.y;
            ss += u.x * u.x + u.y * u.y + v.x * v.x + v.y * v.y;
        }
        ss += __shfl_xor_sync(0xffffffffu, ss, 1);
        ss += __shfl_xor_sync(0xffffffffu, ss, 2);
        if (!live) continue;
        if (w != nullptr) {
            const float rms = 1.f / sqrtf(ss * (1.f / kD) + p.eps);
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const float4 wa = __ldg(reinterpret_cast<const float4 *>(w + 8 * j + e));
                const float4 wb = __ldg(reinterpret_cast<const float4 *>(w + kD / 2 + 8 * j + e));
                x[e] *= rms * wa.x, x[e + 1] *= rms * wa.y, x[e + 2] *= rms * wa.z, x[e + 3] *= rms * wa.w;
                y[e] *= rms * wb.x, y[e + 1] *= rms * wb.y, y[e + 2] *= rms * wb.z, y[e + 3] *= rms * wb.w;
            }
        }
        if (kind < 2) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float o[2], u[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int n = 2 * e + i;
                    o[i] = __fsub_rn(__fmul_rn(x[n], c[n]), __fmul_rn(y[n], s[n]));
                    u[i] = __fadd_rn(__fmul_rn(y[n], c[n]), __fmul_rn(x[n], s[n]));
                }
                aw[e] = pack_bf16(o[0], o[1]);
                bw[e] = pack_bf16(u[0], u[1]);
            }
        }
        *reinterpret_cast<uint4 *>(dst) = make_uint4(aw[0], aw[1], aw[2], aw[3]);
        *reinterpret_cast<uint4 *>(dst + kD / 2) = make_uint4(bw[0], bw[1], bw[2], bw[3]);
    }
}

// ------------------------------------------------------------------ fp8 blocks written and read back
// Where the blocks are: pages, or a ring of `window` cells (block_table null).
struct BlockParams {
    uint8_t *kv;
    const int32_t *block_table, *seq_lens;
    int Hkv, window, max_pages, num_pages, max_seq_len;
};
// The block of positions 16 i .. 16 i + 15 of sequence b and KV head g; null: a page outside the pool.
__device__ __forceinline__ uint8_t *block_of(const BlockParams &p, int b, int i, int g) {
    size_t blk;
    if (p.block_table != nullptr) {
        const int page = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + i);
        if (page < 0 || page >= p.num_pages) {
            flag_status(DA_STATUS_BAD_PAGE);
            return nullptr;
        }
        blk = static_cast<size_t>(page) * p.Hkv + g;
    } else {
        const int per = p.window / kPage;
        blk = (static_cast<size_t>(b) * p.Hkv + g) * per + i % per;
    }
    return p.kv + blk * kBlk8Bytes;
}

__device__ __forceinline__ float fp8_scale(float top, int rule) {
    if (!(top > 0.f)) return 1.f;
    return rule == DA_FP8_SCALE_RECIPROCAL ? __fmul_rn(top, 1.f / 448.f) : __fdiv_rn(top, 448.f);
}

// The new tokens t < n of every sequence quantised into positions L - n + t (a ring keeps the last
// `window` of them). One warp per block that they touch and KV head: lanes 2 t and 2 t + 1 take
// token t of the block, 32 elements of its K row and of its V row each; the V codes are turned
// around through the warp's 1 KiB of shared memory, so that a block that is filled by this call is
// written in whole 16-byte rows. A block that is shared with earlier tokens gets its new bytes only.
constexpr int kStoreWarps = 4;
__global__ void __launch_bounds__(kStoreWarps * 32)
    kv_append_fp8_kernel(const __grid_constant__ BlockParams p, const __nv_bfloat16 *__restrict__ k_new,
                         const __nv_bfloat16 *__restrict__ v_new, const int32_t *__restrict__ q_lens, int T, int rule) {
    __shared__ __align__(16) uint8_t s_v[kStoreWarps][kPage * kD];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    const int L = __ldg(p.seq_lens + b);
    const int n = q_lens != nullptr ? __ldg(q_lens + b) : T;
    bool bad = L < 0 || n < 0 || n > T || (L > 0 && n > L);
    if (p.block_table != nullptr) bad = bad || L > p.max_seq_len || L > static_cast<long long>(p.max_pages) * kPage;
    if (bad) {
        if (threadIdx.x == 0 && blockIdx.x == 0) flag_status(DA_STATUS_BAD_SEQ_LEN);
        return;
    }
    if (L == 0 || n == 0) return;
    const int base = L - n;
    const int lo = p.block_table == nullptr ? max(base, L - p.window) : base;  // the first position stored
    const int unit = blockIdx.x * kStoreWarps + warp;
    const int blk_i = lo / kPage + unit / p.Hkv, g = unit % p.Hkv;
    if (blk_i > (L - 1) / kPage) return;
    uint8_t *blk = block_of(p, b, blk_i, g);
    if (blk == nullptr) return;
    const int t = lane >> 1, half = lane & 1;
    const int pos = blk_i * kPage + t;
    const bool live = pos >= lo && pos < L;
    const uint32_t mask = __ballot_sync(0xffffffffu, live);  // two bits per token
    uint4 raw[2][4];
    if (live) {
        const size_t src = ((static_cast<size_t>(b) * T + (pos - base)) * p.Hkv + g) * kD + 32 * half;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            raw[0][i] = __ldg(reinterpret_cast<const uint4 *>(k_new + src) + i);
            raw[1][i] = __ldg(reinterpret_cast<const uint4 *>(v_new + src) + i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[0][i] = raw[1][i] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        float x[32], top = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w[4] = {raw[kv][i].x, raw[kv][i].y, raw[kv][i].z, raw[kv][i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 u = unpack_bf16(w[e]);
                x[8 * i + 2 * e] = u.x;
                x[8 * i + 2 * e + 1] = u.y;
                top = fmaxf(top, fmaxf(fabsf(u.x), fabsf(u.y)));
            }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        const float scale = fp8_scale(top, rule);
        uint32_t code[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t lo2 = f32x2_to_e4m3x2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale));
            const uint32_t hi2 = f32x2_to_e4m3x2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale));
            code[i] = lo2 | hi2 << 16;
        }
        uint4 *dst = reinterpret_cast<uint4 *>((kv == 0 ? blk : s_v[warp]) + t * kD + 32 * half);
        if (live || kv == 1) {
            dst[0] = make_uint4(code[0], code[1], code[2], code[3]);
            dst[1] = make_uint4(code[4], code[5], code[6], code[7]);
        }
        if (live && half == kv) reinterpret_cast<float *>(blk + kBlk8S)[kv * kPage + t] = scale;
    }
    __syncwarp();
    const uint8_t *sv = s_v[warp];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int d = lane + 32 * i;
        uint8_t *dst = blk + kBlk8V + d * kPage;
        if (mask == 0xffffffffu) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[e] = sv[(4 * e) * kD + d] | sv[(4 * e + 1) * kD + d] << 8 | sv[(4 * e + 2) * kD + d] << 16 |
                       static_cast<uint32_t>(sv[(4 * e + 3) * kD + d]) << 24;
            *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            for (uint32_t m = mask & 0x55555555u; m != 0; m &= m - 1) {
                const int tt = (__ffs(static_cast<int>(m)) - 1) >> 1;
                dst[tt] = sv[tt * kD + d];
            }
        }
    }
}

// Positions first .. L - 1 (first = starts[b], or 0; at most N of them) of every sequence as bf16
// rows i = position - first of k_out / v_out [B][N][Hkv][64]: e4m3(code) times the token's scale in
// fp32, rounded to bf16. Rows past them are not written. One warp per block and KV head, the V
// codes turned around through shared memory. Positions that a ring has dropped are not there to
// be read: DA_STATUS_BAD_SEQ_LEN. wide: both outputs start at 32-byte addresses (then one store takes
// a lane's 16 elements).
__global__ void __launch_bounds__(kStoreWarps * 32)
    kv_read_fp8_kernel(const __grid_constant__ BlockParams p, const int32_t *__restrict__ starts, int N,
                       __nv_bfloat16 *__restrict__ k_out, __nv_bfloat16 *__restrict__ v_out, int wide) {
    __shared__ __align__(16) uint8_t s_v[kStoreWarps][kPage * kD];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    const int L = __ldg(p.seq_lens + b);
    const int first = starts != nullptr ? __ldg(starts + b) : 0;
    bool bad = L < 0 || first < 0 || first > L;
    if (p.block_table != nullptr)
        bad = bad || L > p.max_seq_len || L > static_cast<long long>(p.max_pages) * kPage;
    else
        bad = bad || first < L - p.window;
    if (bad) {
        if (threadIdx.x == 0 && blockIdx.x == 0) flag_status(DA_STATUS_BAD_SEQ_LEN);
        return;
    }
    const int end = static_cast<int>(min(static_cast<long long>(L), static_cast<long long>(first) + N));
    const int unit = blockIdx.x * kStoreWarps + warp;
    const int blk_i = first / kPage + unit / p.Hkv, g = unit % p.Hkv;
    if (first >= end || blk_i > (end - 1) / kPage) return;
    const uint8_t *blk = block_of(p, b, blk_i, g);
    if (blk == nullptr) return;
    uint4 kc[2], vc[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        kc[i] = *(reinterpret_cast<const uint4 *>(blk) + lane + 32 * i);
        vc[i] = *(reinterpret_cast<const uint4 *>(blk + kBlk8V) + lane + 32 * i);
    }
    const float sc = *(reinterpret_cast<const float *>(blk + kBlk8S) + lane);  // K scales, then V scales
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t w[4] = {vc[i].x, vc[i].y, vc[i].z, vc[i].w};
#pragma unroll
        for (int t = 0; t < kPage; ++t) s_v[warp][t * kD + lane + 32 * i] = static_cast<uint8_t>(w[t >> 2] >> (8 * (t & 3)));
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) vc[i] = reinterpret_cast<const uint4 *>(s_v[warp])[lane + 32 * i];
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // token t, elements 16 (lane % 4) .. + 15
        const int t = (lane >> 2) + 8 * i, pos = blk_i * kPage + t;
        const float ks = __shfl_sync(0xffffffffu, sc, t), vs = __shfl_sync(0xffffffffu, sc, kPage + t);
        if (pos < first || pos >= end) continue;
        const size_t row = ((static_cast<size_t>(b) * N + (pos - first)) * p.Hkv + g) * kD + 16 * (lane & 3);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint4 c = kv == 0 ? kc[i] : vc[i];
            const float s = kv == 0 ? ks : vs;
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t h[2];
                e4m3x4_to_f16x2x2(w[e], h[0], h[1]);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[u]));
                    o[2 * e + u] = pack_bf16(f.x * s, f.y * s);
                }
            }
            __nv_bfloat16 *dst = (kv == 0 ? k_out : v_out) + row;
            if (wide) {
                st_global_v8(dst, o);
            } else {
                reinterpret_cast<uint4 *>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
                reinterpret_cast<uint4 *>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
            }
        }
    }
}
