// What stands around the attention over an fp8 cache in a step of new tokens: the norms and the
// rotation of the projected queries and keys (qk_norm_rope_kernel), the tokens quantised into
// their blocks (kv_append_fp8_kernel), and cached positions read back as bf16
// (kv_read_fp8_kernel).
//
// Included into decode_attn.cu (inside its anonymous namespace): one translation unit, sharing
// the fp8 helpers and the status word.

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// ------------------------------------------------------------------ norms and rotation
// Row x of 64 values of one head: y = x w / sqrt(sum(x^2) / 64 + eps) (no norm: y = x), then the
// pairs (i, i + 32) rotated by row pos[axis(i)] of the tables. All in fp32, rounded once to bf16;
// the rotation's products and its sum or difference are rounded one by one, as in the other
// calls with a rotary embedding (without a norm the bits are theirs).
//
// Every row is read and written once. Four lanes hold a row, lane j its elements 8 j .. + 7 and
// 32 + 8 j .. + 7, so that a lane has both halves of its pairs (two 16-byte loads and stores, no exchange for the
// rotation; two shuffles for the norm). A warp takes eight rows of a token at a time; a lane keeps its pairs' cosines
// and sines over all of them, with a norm multiplied by the head's weights once: the pair is then
//     r (x (c w_x) - y (s w_y)),  r (y (c w_y) + x (s w_x)),   r = 1 / sqrt(..),
// two values per instruction (240 instructions per eight rows had bound the kernel, not memory: 8191 tokens of 80 rows
// took 36.6 us). The rows come through shared memory, four eights ahead: registers had limited the loads in flight
// (37.7 us). 31.3 us back to back, 5.4 TB/s of the 6.7 of a plain copy.
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
constexpr int kRotAhead = 4;  // eights of rows on their way
// Warps per SM that a token's rows are spread over where there are few tokens: with 8 / 16 / 32, 64 tokens of 80 rows took
// 6.2 / 6.2 / 8.1 us (events around one call), 1024 12.3 each, 2432 16.4 / 16.4 / 18.4.
constexpr int kRotWarps = 16;

// Rows h0 + lane / 4, + 8, .. below h1 of one token's query or key heads (in and out at head 0, this lane's first
// element). c, s: the lane's pairs' angles, two pairs each; w: the heads' norm weights from this lane's first element on.
template <bool NORM>
__device__ __forceinline__ void rotate_rows(const __nv_bfloat16 *in, __nv_bfloat16 *out, int h0, int h1, const float2 (&c)[4],
                                            const float2 (&s)[4], const float *w, float eps, int lane, uint8_t *stage) {
    // coefficients of x and y in both results
    float2 xc[4], ys[4], yc[4], xs[4];
    if (NORM)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 wx = __ldg(reinterpret_cast<const float2 *>(w) + e), wy = __ldg(reinterpret_cast<const float2 *>(w + kD / 2) + e);
            xc[e] = mul2(c[e], wx);
            xs[e] = mul2(s[e], wx);
            yc[e] = mul2(c[e], wy);
            ys[e] = mul2(make_float2(-s[e].x, -s[e].y), wy);
        }
    const float2 one = make_float2(1.f, 1.f);
    in += (h0 + (lane >> 2)) * kD;
    out += (h0 + (lane >> 2)) * kD;
    // this lane's 32 bytes of the rows kRotAhead eights ahead, copied into its own places of shared memory
    const uint32_t mine = smem_addr(stage) + 16 * lane;
    auto fetch = [&](int k) {
        if (h0 + 8 * k + (lane >> 2) < h1) {
            const uint32_t dst = mine + k % kRotAhead * 1024;
            const __nv_bfloat16 *src = in + 8 * k * kD;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 512), "l"(src + kD / 2) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int k = 0; k < kRotAhead - 1; ++k) fetch(k);
    for (int k = 0; h0 + 8 * k < h1; ++k, out += 8 * kD) {  // (all lanes stay for the shuffles)
        const bool live = h0 + 8 * k + (lane >> 2) < h1;
        fetch(k + kRotAhead - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kRotAhead - 1) : "memory");
        const uint4 a = *reinterpret_cast<const uint4 *>(stage + k % kRotAhead * 1024 + 16 * lane);
        const uint4 b = *reinterpret_cast<const uint4 *>(stage + k % kRotAhead * 1024 + 512 + 16 * lane);
        uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
        float2 x[4], y[4], r = one;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[e] = unpack_bf16(aw[e]);
            y[e] = unpack_bf16(bw[e]);
        }
        if (NORM) {
            float2 q = mul2(x[0], x[0]);
#pragma unroll
            for (int e = 1; e < 4; ++e) q = fma2(x[e], x[e], q);
#pragma unroll
            for (int e = 0; e < 4; ++e) q = fma2(y[e], y[e], q);
            float ss = q.x + q.y;
            ss += __shfl_xor_sync(0xffffffffu, ss, 1);
            ss += __shfl_xor_sync(0xffffffffu, ss, 2);
            r.x = r.y = rsqrtf(ss * (1.f / kD) + eps);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float2 o, u;
            if (NORM) {
                o = mul2(r, fma2(x[e], xc[e], mul2(y[e], ys[e])));
                u = mul2(r, fma2(y[e], yc[e], mul2(x[e], xs[e])));
            } else {  // every product and sum rounded by itself
                o = make_float2(__fsub_rn(__fmul_rn(x[e].x, c[e].x), __fmul_rn(y[e].x, s[e].x)),
                                __fsub_rn(__fmul_rn(x[e].y, c[e].y), __fmul_rn(y[e].y, s[e].y)));
                u = make_float2(__fadd_rn(__fmul_rn(y[e].x, c[e].x), __fmul_rn(x[e].x, s[e].x)),
                                __fadd_rn(__fmul_rn(y[e].y, c[e].y), __fmul_rn(x[e].y, s[e].y)));
            }
            aw[e] = pack_bf16(o.x, o.y);
            bw[e] = pack_bf16(u.x, u.y);
        }
        if (live) {
            *reinterpret_cast<uint4 *>(out) = make_uint4(aw[0], aw[1], aw[2], aw[3]);
            *reinterpret_cast<uint4 *>(out + kD / 2) = make_uint4(bw[0], bw[1], bw[2], bw[3]);
        }
    }
}

__global__ void __launch_bounds__(kRotThreads) qk_norm_rope_kernel(const __grid_constant__ RotateParams p) {
    __shared__ __align__(16) uint8_t s_rows[kRotThreads / 32][kRotAhead * 1024];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunks = (p.rows + p.chunk - 1) / p.chunk;
    const long long item = static_cast<long long>(blockIdx.x) * (kRotThreads / 32) + warp;
    const long long tok = item / chunks;
    if (tok >= p.N) return;
    const int r0 = static_cast<int>(item - tok * chunks) * p.chunk, r1 = min(r0 + p.chunk, p.rows);
    const int j = lane & 3, Hqk = p.Hq + p.Hkv;
    if (r0 < Hqk) {
        float2 c[4], s[4];
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
            float cv[4], sv[4];
            if (p.quads >> (i0 >> 2) & 1) {
                const size_t at = row_of(p.axis[i0]) + i0;
                const float4 c4 = __ldg(reinterpret_cast<const float4 *>(p.rope_cos + at));
                const float4 s4 = __ldg(reinterpret_cast<const float4 *>(p.rope_sin + at));
                cv[0] = c4.x, cv[1] = c4.y, cv[2] = c4.z, cv[3] = c4.w;
                sv[0] = s4.x, sv[1] = s4.y, sv[2] = s4.z, sv[3] = s4.w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const size_t at = row_of(p.axis[i0 + e]) + i0 + e;
                    cv[e] = __ldg(p.rope_cos + at);
                    sv[e] = __ldg(p.rope_sin + at);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                c[2 * h + e] = make_float2(cv[2 * e], cv[2 * e + 1]);
                s[2 * h + e] = make_float2(sv[2 * e], sv[2 * e + 1]);
            }
        }
        if (bad) flag_status(DA_STATUS_BAD_POSITION);
        auto rows = [&](const __nv_bfloat16 *in, __nv_bfloat16 *out, int h0, int h1, const float *w) {
            if (h0 >= h1) return;
            if (w != nullptr)
                rotate_rows<true>(in + 8 * j, out + 8 * j, h0, h1, c, s, w + 8 * j, p.eps, lane, s_rows[warp]);
            else
                rotate_rows<false>(in + 8 * j, out + 8 * j, h0, h1, c, s, nullptr, 0.f, lane, s_rows[warp]);
        };
        rows(p.q + tok * p.q_ld, p.q_out + tok * p.qo_ld, r0, min(r1, p.Hq), p.q_weight);
        rows(p.k + tok * p.k_ld, p.k_out + tok * p.ko_ld, max(r0 - p.Hq, 0), min(r1 - p.Hq, p.Hkv), p.k_weight);
    }
    for (int h = max(r0 - Hqk, 0) + (lane >> 3); h < r1 - Hqk; h += 4)  // value rows, eight lanes each
        reinterpret_cast<uint4 *>(p.v_out + tok * p.vo_ld + h * kD)[lane & 7] = reinterpret_cast<const uint4 *>(p.v + tok * p.v_ld + h * kD)[lane & 7];
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

// x / scale of a row, correctly rounded: the quotient's first guess x r, r = RN(1 / scale), corrected by its exact
// remainder, is the rounded quotient (Markstein's theorem, IBM J. Res. Dev. 34, 1990), as long as nothing under- or
// overflows on the way. Rows whose largest magnitude lies far from both ends of fp32's range qualify: their scale and
// its reciprocal are normal, and a remainder can only be inexact where the quotient is far below half of e4m3's
// smallest step, 2^-10. The others divide. Three operations, two values at a time, instead of a division's ten or so: with
// divisions, their branches and V^T written byte by byte the kernel took 51 us for 42000 tokens of 8 heads, now 34.
struct RowScale {
    float scale, r;
    bool fast;
    __device__ __forceinline__ RowScale(float top, int rule) {
        scale = fp8_scale(top, rule);
        fast = top >= 1e-20f && top <= 1e30f;
        r = fast ? __frcp_rn(scale) : 0.f;
    }
    __device__ __forceinline__ float2 quotients(float2 x) const {
        const float2 q = mul2(x, make_float2(r, r)), d = fma2(q, make_float2(scale, scale), make_float2(-x.x, -x.y));
        return fma2(make_float2(-d.x, -d.y), make_float2(r, r), q);  // (the remainder's negative: so that -0 stays -0)
    }
};
// Four values to e4m3 codes (nearest, ties to even, saturating at +-448; NaN: 0x7f), low byte first.
__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(float2 a, float2 b) {
    uint32_t d;
    asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(d)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// Eight bf16 values of a row (16 bytes) to their codes.
__device__ __forceinline__ uint2 fp8_codes8(const uint4 &v, const RowScale &s) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float2 q[4];
    if (s.fast) {
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = s.quotients(unpack_bf16(w[e]));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = unpack_bf16(w[e]);
            q[e] = make_float2(__fdiv_rn(f.x, s.scale), __fdiv_rn(f.y, s.scale));
        }
    }
    return make_uint2(f32x4_to_e4m3x4(q[0], q[1]), f32x4_to_e4m3x4(q[2], q[3]));
}
// The larger magnitudes of two pairs of bf16 values, of whatever sign (a NaN loses against a number, as in fmaxf).
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t w) {
    uint32_t d;
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(m), "r"(w));
    return d;
}
// Four words of four bytes, turned around: word i of the result holds byte i of each.
__device__ __forceinline__ void transpose4x4(uint32_t (&w)[4]) {
    const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[0], w[1], 0x7362);
    const uint32_t c = __byte_perm(w[2], w[3], 0x5140), d = __byte_perm(w[2], w[3], 0x7362);
    w[0] = __byte_perm(a, c, 0x5410);
    w[1] = __byte_perm(a, c, 0x7632);
    w[2] = __byte_perm(b, d, 0x5410);
    w[3] = __byte_perm(b, d, 0x7632);
}

// The new tokens t < n of every sequence quantised into positions L - n + t (a ring keeps the last
// `window` of them). One warp per block that they touch and KV head: lane 4 t' + j takes elements
// 8 j .. + 7 and 32 + 8 j .. + 7 of tokens t' and t' + 8 of the block, so that every load and every store of codes is
// made of whole sectors. The V codes are turned around, four by four bytes, on their way through the warp's shared
// memory; a block that is filled by this call is written in whole words, one that is shared with earlier tokens
// gets its new bytes only. 42000 tokens of 8 heads: 34 us for 132 MB, 20 at
// the memory's rate; DRAM and arithmetic are both near half (2.4 instructions a cycle), the rest is each warp's chain of
// load, maximum, quotients, exchange and store. clear: counters of the attention that follows in the same call (multi_tc8_kernel).
constexpr int kStoreWarps = 4;
constexpr int kCodePitch = 72;  // bytes from one token's codes to the next: the turning reads meet no bank twice
__global__ void __launch_bounds__(kStoreWarps * 32)
    kv_append_fp8_kernel(const __grid_constant__ BlockParams p, const __nv_bfloat16 *__restrict__ k_new,
                         const __nv_bfloat16 *__restrict__ v_new, const int32_t *__restrict__ q_lens, int T, int rule,
                         int *clear, int n_clear) {
    __shared__ __align__(16) uint8_t s_v[kStoreWarps][kPage * kCodePitch];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    if (blockIdx.x == 0 && b == 0)
        for (int i = threadIdx.x; i < n_clear; i += blockDim.x) clear[i] = 0;
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
    const int first = p.block_table == nullptr ? max(base, L - p.window) : base;  // the first position stored
    const int unit = blockIdx.x * kStoreWarps + warp;
    const int blk_i = first / kPage + unit / p.Hkv, g = unit % p.Hkv;
    if (blk_i > (L - 1) / kPage) return;
    const int pos0 = blk_i * kPage, t_lo = max(0, first - pos0), t_hi = min(kPage, L - pos0);  // tokens [t_lo, t_hi)
    const int t = lane >> 2, j = lane & 3;
    uint4 raw[2][2][2];  // K, V; token t, t + 8; elements 8 j, 32 + 8 j
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int tt = t + 8 * h;
        const bool live = tt >= t_lo && tt < t_hi;
        const size_t src = ((static_cast<size_t>(b) * T + (pos0 + tt - base)) * p.Hkv + g) * kD + 8 * j;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            raw[0][h][i] = live ? __ldg(reinterpret_cast<const uint4 *>(k_new + src + 32 * i)) : make_uint4(0, 0, 0, 0);
            raw[1][h][i] = live ? __ldg(reinterpret_cast<const uint4 *>(v_new + src + 32 * i)) : make_uint4(0, 0, 0, 0);
        }
    }
    uint8_t *blk = block_of(p, b, blk_i, g);  // (read while the rows are on their way)
    if (blk == nullptr) return;
    uint8_t *sv = s_v[warp];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int tt = t + 8 * h;
            const bool live = tt >= t_lo && tt < t_hi;
            const uint4 &a = raw[kv][h][0], &c = raw[kv][h][1];
            uint32_t m = abs_max2(abs_max2(a.x, a.y), abs_max2(a.z, a.w));
            m = abs_max2(m, abs_max2(abs_max2(c.x, c.y), abs_max2(c.z, c.w)));
            m = abs_max2(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = abs_max2(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const float2 top = unpack_bf16(m);
            const RowScale rs(fmaxf(fabsf(top.x), fabsf(top.y)), rule);
            const uint2 ca = fp8_codes8(a, rs), cc = fp8_codes8(c, rs);
            if (kv == 0) {
                if (live) {
                    *reinterpret_cast<uint2 *>(blk + tt * kD + 8 * j) = ca;
                    *reinterpret_cast<uint2 *>(blk + tt * kD + 32 + 8 * j) = cc;
                }
            } else {
                *reinterpret_cast<uint2 *>(sv + tt * kCodePitch + 8 * j) = ca;
                *reinterpret_cast<uint2 *>(sv + tt * kCodePitch + 32 + 8 * j) = cc;
            }
            if (live && j == 0) reinterpret_cast<float *>(blk + kBlk8S)[kv * kPage + tt] = rs.scale;
        }
    __syncwarp();
    if (t_lo == 0 && t_hi == kPage) {  // elements 4 (lane % 16) .. + 3 of tokens 8 (lane / 16) .. + 7
        const int dq = lane & 15, th = lane >> 4;
        uint32_t w[2][4];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i >> 2][i & 3] = *reinterpret_cast<const uint32_t *>(sv + (8 * th + i) * kCodePitch + 4 * dq);
        transpose4x4(w[0]);
        transpose4x4(w[1]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint2 *>(blk + kBlk8V + (4 * dq + e) * kPage + 8 * th) = make_uint2(w[0][e], w[1][e]);
    } else {
        for (int tt = t_lo; tt < t_hi; ++tt)
#pragma unroll
            for (int i = 0; i < 2; ++i) blk[kBlk8V + (lane + 32 * i) * kPage + tt] = sv[tt * kCodePitch + lane + 32 * i];
    }
}

// Eight codes times their token's scale as bf16.
__device__ __forceinline__ uint4 fp8_values8(uint2 c, float s) {
    const uint32_t w[2] = {c.x, c.y};
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        uint32_t h[2];
        e4m3x4_to_f16x2x2(w[e], h[0], h[1]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[u]));
            o[2 * e + u] = pack_bf16(f.x * s, f.y * s);
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Positions first .. L - 1 (first = starts[b], or 0; at most N of them) of every sequence as bf16
// rows i = position - first of k_out / v_out [B][N][Hkv][64]: e4m3(code) times the token's scale in
// fp32, rounded to bf16. Rows past them are not written. One warp per block and KV head; eight lanes
// write a row. The V codes pass through shared memory as they are (a row's 16 tokens every 16 bytes, and 16 bytes more
// every eight rows, so that the reads of eight rows' words meet no bank twice) and are turned around four by four.
// Positions that a ring has dropped are not there to be read: DA_STATUS_BAD_SEQ_LEN.
// 131072 positions of 8 heads, 512 of them appended before: 67 us for 412 MB, 62 at the rate of a plain copy.
__global__ void __launch_bounds__(kStoreWarps * 32)
    kv_read_fp8_kernel(const __grid_constant__ BlockParams p, const int32_t *__restrict__ starts, int N,
                       __nv_bfloat16 *__restrict__ k_out, __nv_bfloat16 *__restrict__ v_out) {
    __shared__ __align__(16) uint8_t s_v[kStoreWarps][(kD + kD / 8) * kPage];
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
    const int pos0 = blk_i * kPage, o = lane & 7;  // elements 8 o .. + 7
    uint2 kc[4];
    uint4 vc[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) kc[i] = *(reinterpret_cast<const uint2 *>(blk) + lane + 32 * i);  // token lane / 8 + 4 i
#pragma unroll
    for (int i = 0; i < 2; ++i) vc[i] = *(reinterpret_cast<const uint4 *>(blk + kBlk8V) + lane + 32 * i);
    const float sc = *(reinterpret_cast<const float *>(blk + kBlk8S) + lane);  // K scales, then V scales
    uint8_t *sv = s_v[warp];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int d = lane + 32 * i;
        *reinterpret_cast<uint4 *>(sv + (d + (d >> 3)) * kPage) = vc[i];
    }
    auto row = [&](int t) { return ((static_cast<size_t>(b) * N + (pos0 + t - first)) * p.Hkv + g) * kD + 8 * o; };
    auto there = [&](int t) { return pos0 + t >= first && pos0 + t < end; };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = (lane >> 3) + 4 * i;
        const float s = __shfl_sync(0xffffffffu, sc, t);
        if (there(t)) *reinterpret_cast<uint4 *>(k_out + row(t)) = fp8_values8(kc[i], s);
    }
    __syncwarp();
    const int t4 = lane >> 3;  // tokens 4 t4 .. + 3
    uint32_t w[2][4];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e >> 2][e & 3] = *reinterpret_cast<const uint32_t *>(sv + (8 * o + e + o) * kPage + 4 * t4);
    transpose4x4(w[0]);
    transpose4x4(w[1]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = 4 * t4 + i;
        const float s = __shfl_sync(0xffffffffu, sc, kPage + t);
        if (there(t)) *reinterpret_cast<uint4 *>(v_out + row(t)) = fp8_values8(make_uint2(w[0][i], w[1][i]), s);
    }
}
