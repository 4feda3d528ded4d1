// Accumulated attention weights: after the attention of a step each attended cell gets the sum of
// its probabilities over the query rows of its KV head,
//     w[cell(j)] += sum_r 2^(s_rj - lse_r),     rows r = t G + h that see j,
// with s the scores in log2 units and lse_r log2 of row r's softmax denominator, which the
// attention kernels leave in p.nlse (negated). The cell of a token appended by the call gets the
// sum alone. A cell's sum is made by fixed threads in a fixed order and added with one
// reduction, so nothing depends on an order except the additions of several sequences to a
// page they share.
//
// One token per sequence: the attention kernel leaves its scores too (score_weights_kernel below
// reads them back, mostly from L2). Several tokens: the scores are formed again on the tensor
// cores (multi_weights_kernel), since T times as many would cost more to write and read than
// the keys cost to read.

struct WeightParams {
    float *weights;                  // [num_pages][Hkv][16]
    const int *block_table, *seq_lens, *q_lens;
    const float *nlse;               // [B * Hkv][lse_ld]
    int lse_ld;
    const float *scores;             // one token: [unit][16][G]
    float scale_log2;
    int B, Hkv, G, T, window, max_pages, num_pages, max_seq_len;
    int assign_new;                  // the call appended its new tokens
    int run;                         // several tokens: 128-key stages per CTA
};

// ------------------------------------------------------------------ one token per sequence
// Warps take equal contiguous shares of the call's units (16-token tiles in the attention
// kernel's order), 32 at a time: lane l works out the address of the batch's unit l, then the
// warp takes the units four at a time, two lanes per token and half its heads each.
constexpr int kSwThreads = 256;
constexpr int kSwCtasPerSm = 4;

template <int K>
__device__ __forceinline__ void load_floats(float (&v)[K], const float *p) {
    if constexpr (K >= 4) {
#pragma unroll
        for (int i = 0; i < K / 4; ++i) {
            const float4 x = reinterpret_cast<const float4 *>(p)[i];
            v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
        }
    } else if constexpr (K == 2) {
        const float2 x = *reinterpret_cast<const float2 *>(p);
        v[0] = x.x; v[1] = x.y;
    } else {
        v[0] = *p;
    }
}

template <int G>
__global__ void __launch_bounds__(kSwThreads, kSwCtasPerSm) score_weights_kernel(const WeightParams p) {
    constexpr int HPL = G > 1 ? G / 2 : 1;    // heads per lane
    constexpr int kSwUnroll = G > 8 ? 2 : 4;  // tiles in flight (64 registers)
    __shared__ int s_pre[kMaxBatch + 1], s_len[kMaxBatch], s_wsum[kSwThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int B = p.B, Hkv = p.Hkv;
    // The lengths were read by the attention kernel just before this one, after its own wait, so
    // they are final before this grid may start: the prefix is worked out before the wait.
    {
        int v[4], tsum = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int b = tid * 4 + k;
            int L = b < B ? __ldg(p.seq_lens + b) : 0;
            if (L < 0 || L > p.max_seq_len || L > p.max_pages * kPage) L = 0;  // (flagged by the attention)
            if (b < B) s_len[b] = L;
            v[k] = tiles_of<false>(L, p.window) * Hkv;
            tsum += v[k];
        }
        int incl = tsum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        if (lane == 31) s_wsum[warp] = incl;
        __syncthreads();
        int run = incl - tsum;
        for (int w = 0; w < warp; ++w) run += s_wsum[w];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int b = tid * 4 + k;
            if (b < B) s_pre[b] = run;
            run += v[k];
        }
        if (tid == kSwThreads - 1) s_pre[B] = run;
        __syncthreads();
    }
    const int U = s_pre[B];
    const long long nw = static_cast<long long>(gridDim.x) * (kSwThreads / 32);
    const long long w = static_cast<long long>(blockIdx.x) * (kSwThreads / 32) + warp;
    const int ua = static_cast<int>(U * w / nw), ue = static_cast<int>(U * (w + 1) / nw);
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int tok = G > 1 ? lane >> 1 : lane;             // this lane's token of a tile (G = 1: lanes 0-15)
    const int off = G > 1 ? lane * HPL : lane;            // its scores in the tile, and its heads
    const int hoff = G > 1 ? (lane & 1) * HPL : 0;
    for (int u0 = ua; u0 < ue; u0 += 32) {
        // lane l: cells of unit u0 + l (-1: bad page), its denominators, its attended tokens
        // [lo, hi) and the token appended by this call (16: none)
        int cell = -1, bg = 0, range = 0;
        if (u0 + lane < ue) {
            const int x = u0 + lane;
            const int b = find_seq(s_pre, B, x);
            const int tiles = (s_pre[b + 1] - s_pre[b]) / Hkv, r = x - s_pre[b];
            const int g = r / tiles, t = r - g * tiles;
            const int L = s_len[b], lo = (p.window > 0 && L > p.window) ? L - p.window : 0;
            const int pt = lo / kPage + t;
            const int page = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + pt);
            if (page >= 0 && page < p.num_pages) cell = page * Hkv + g;
            bg = b * Hkv + g;
            const int fresh = p.assign_new ? L - 1 - pt * kPage : 16;
            range = max(0, lo - pt * kPage) | (min(16, L - pt * kPage) << 8) | (min(fresh, 16) << 16);
        }
        const int cnt = min(32, ue - u0);
        for (int i = 0; i < cnt; i += kSwUnroll) {
            float s[kSwUnroll][HPL], l[kSwUnroll][HPL];
            int c[kSwUnroll], rg[kSwUnroll];
#pragma unroll
            for (int k = 0; k < kSwUnroll; ++k) {
                const int src = min(i + k, cnt - 1);
                c[k] = __shfl_sync(0xffffffffu, cell, src);
                rg[k] = __shfl_sync(0xffffffffu, range, src);
                const int bgk = __shfl_sync(0xffffffffu, bg, src);
                if (i + k >= cnt || (G == 1 && lane >= 16)) c[k] = -1;
                if (c[k] >= 0) {
                    load_floats(s[k], p.scores + static_cast<size_t>(u0 + i + k) * (kPage * G) + off);
                    load_floats(l[k], p.nlse + static_cast<size_t>(bgk) * G + hoff);
                }
            }
#pragma unroll
            for (int k = 0; k < kSwUnroll; ++k) {
                float sum = 0.f;
                if (c[k] >= 0)
#pragma unroll
                    for (int h = 0; h < HPL; ++h) sum += fast_exp2(s[k][h] + l[k][h]);
                if (G > 1) sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                const int lo = rg[k] & 255, hi = (rg[k] >> 8) & 255, fresh = rg[k] >> 16;
                if (c[k] >= 0 && tok >= lo && tok < hi && (G == 1 || (lane & 1) == 0)) {
                    float *dst = p.weights + static_cast<size_t>(c[k]) * kPage + tok;
                    if (tok == fresh)
                        *dst = sum;
                    else
                        atomicAdd(dst, sum);
                }
            }
        }
    }
}

// ------------------------------------------------------------------ several tokens per sequence
// One CTA per (sequence, KV head, run of 128-key stages). S^T = K Q^T on tcgen05 puts the keys on
// the TMEM lanes (M = 128) and N query rows on the columns, so a key's sum over the rows is a sum
// along a thread's own columns: no shuffles, and the denominators are the same for every lane (one
// broadcast shared-memory read per four columns). Ten warps:
//   warps 0-7  columns [0, N/2) (warps 0-3) and [N/2, N) (4-7) of the stage's 128 keys: exponentials
//              and sums, into shared memory per (stage, half, key)
//   warp 8     TMA: key stages (8 tiles), query blocks with their denominators
//   warp 9     MMA issue, two TMEM buffers of N columns
// Up to 256 rows (N = 32, 64, 128, 256): one query block stays, the key stages stream through a
// ring. More: the run's stages (at most kMwResident) stay, and query blocks of 256 rows stream
// through two slots; a key's sum then takes several blocks, added with a compensated sum (16384
// terms one after another in 32 bits would lose the last bits).
// Blocks of rows that see no key of a stage (causal mask, window) are skipped by every role.
constexpr int kMwKeys = 128;
constexpr int kMwTiles = kMwKeys / kPage;
constexpr int kMwKBytes = kMwKeys * kD * 2;  // 16 KiB per key stage
constexpr int kMwMaxRows = 256;              // query rows per block
constexpr int kMwResident = 4;               // key stages per CTA when query blocks stream
constexpr int kMwMaxRun = 16;                // key stages per CTA at most
constexpr int kMwThreads = 320;

template <int N>
struct MwLayout {
    static constexpr int kQSlots = N == kMwMaxRows ? 2 : 1;
    static constexpr int kRing = N == kMwMaxRows ? 6 : 4;
    static constexpr int kQBytes = N * kD * 2;
    static constexpr int k = kQSlots * kQBytes;
    static constexpr int lse = k + kRing * kMwKBytes;
    static constexpr int acc = lse + kQSlots * N * 4;
    static constexpr int bars = acc + kMwMaxRun * 2 * kMwKeys * 4;
    static constexpr int kBars = 2 * kRing + 2 * kQSlots + 5;
    static constexpr int bytes = 1024 + bars + kBars * 8;  // with the slack to align the base
    static constexpr int kCtas = N == kMwMaxRows ? 1 : 2;  // resident per SM
    static_assert(kQBytes % 1024 == 0 && acc % 16 == 0 && bars % 8 == 0, "alignment");
    static_assert(kCtas * (bytes + 1024) <= 233472, "shared memory of the CTAs on one SM");
    static_assert(kMwResident <= kRing && kMwResident * 2 <= kMwMaxRun, "resident stages, compensated sums");
};

__device__ __forceinline__ void tma_load_3d_plain(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2,
                                                  uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Sum of 2^(x scale + nlse) over CH columns; columns outside [lo, hi) left out if MASK.
template <int CH, bool MASK>
__device__ __forceinline__ float sum_columns(const uint32_t (&v)[CH], const float *nlse, float scale, int lo, int hi) {
    float2 acc[2] = {{0.f, 0.f}, {0.f, 0.f}};
    const float2 sc = make_float2(scale, scale);
#pragma unroll
    for (int c = 0; c < CH; c += 4) {
        const float4 l = *reinterpret_cast<const float4 *>(nlse + c);
        const float2 x = fma2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), sc, make_float2(l.x, l.y));
        const float2 y = fma2(make_float2(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])), sc, make_float2(l.z, l.w));
        float2 ex = make_float2(fast_exp2(x.x), fast_exp2(x.y)), ey = make_float2(fast_exp2(y.x), fast_exp2(y.y));
        if (MASK) {
            ex.x = c >= lo && c < hi ? ex.x : 0.f;
            ex.y = c + 1 >= lo && c + 1 < hi ? ex.y : 0.f;
            ey.x = c + 2 >= lo && c + 2 < hi ? ey.x : 0.f;
            ey.y = c + 3 >= lo && c + 3 < hi ? ey.y : 0.f;
        }
        acc[0] = add2(acc[0], ex);
        acc[1] = add2(acc[1], ey);
    }
    return (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
}

template <int N>
__global__ void __launch_bounds__(kMwThreads, MwLayout<N>::kCtas)
    multi_weights_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmq,
                         const WeightParams p) {
    using Lay = MwLayout<N>;
    constexpr int kRing = Lay::kRing, kQSlots = Lay::kQSlots;
    constexpr int kHalf = N / 2, CH = kHalf < 32 ? 16 : 32;  // columns per warp, and per TMEM load
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t q_s = smem_addr(smem), k_s = q_s + Lay::k;
    float *const s_lse = reinterpret_cast<float *>(smem + Lay::lse);
    float *const s_acc = reinterpret_cast<float *>(smem + Lay::acc);
    const uint32_t k_full = smem_addr(smem + Lay::bars), k_empty = k_full + 8 * kRing;
    const uint32_t q_full = k_empty + 8 * kRing, q_empty = q_full + 8 * kQSlots;
    const uint32_t t_full = q_empty + 8 * kQSlots, t_empty = t_full + 16, drain = t_empty + 16;
    __shared__ uint32_t s_tmem;
    __shared__ int s_failed;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = blockIdx.y, b = blockIdx.z;
    if (tid == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmk)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmq)) : "memory");
        for (int s = 0; s < kRing; ++s) {
            mbar_init(k_full + 8 * s, 1);
            mbar_init(k_empty + 8 * s, 1);
        }
        for (int s = 0; s < kQSlots; ++s) {
            mbar_init(q_full + 8 * s, 1);
            mbar_init(q_empty + 8 * s, 9);  // the products, and the eight warps that read the denominators
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(t_full + 8 * s, 1);
            mbar_init(t_empty + 8 * s, 8);
        }
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s_failed = 0;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- this CTA's rows and keys (counts out of range were flagged by the attention)
    const int L = __ldg(p.seq_lens + b);
    const int n = p.q_lens != nullptr ? __ldg(p.q_lens + b) : p.T;
    if (L <= 0 || L > p.max_seq_len || L > p.max_pages * kPage || n <= 0 || n > p.T || n > L) return;
    const int base = L - n, W = p.window;
    const int lo0 = W > 0 ? max(0, base - W + 1) : 0;
    const int s0 = lo0 / kMwKeys + blockIdx.x * p.run;     // first stage: positions 128 s0 on
    const int ns = min(p.run, (L - 1) / kMwKeys - s0 + 1);
    if (ns <= 0) return;
    const int nqb = (n * p.G + N - 1) / N;
    const bool many = nqb > 1;                             // query blocks stream, the stages stay
    // does a row of block qb see a key at a position in [first, last]?
    auto sees = [&](int qb, int first, int last) {
        const int t0 = qb * N / p.G, t1 = min(n - 1, (qb * N + N - 1) / p.G);
        return base + t1 >= first && (W == 0 || base + t0 - W + 1 <= last);
    };
    auto sees_stage = [&](int qb, int st) {
        const int first = (s0 + st) * kMwKeys;
        return sees(qb, first, min(first + kMwKeys, L) - 1);
    };
    auto sees_run = [&](int qb) { return sees(qb, s0 * kMwKeys, min((s0 + ns) * kMwKeys, L) - 1); };

    if (many)
        for (int i = tid; i < ns * 2 * kMwKeys; i += kMwThreads) reinterpret_cast<float2 *>(s_acc)[i] = make_float2(0.f, 0.f);
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)),
                     "r"(static_cast<uint32_t>(2 * N)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tmem;
    const size_t bg = static_cast<size_t>(b) * p.Hkv + g;

    bool failed = false;
    if (warp == 8) {
        // ---- TMA: the whole warp; lane u issues tile u of a key stage
        const uint64_t policy = evict_first_policy();
        int ki = 0, qi = 0;  // key stages and query blocks issued
        auto wait_all = [&](uint32_t bar, uint32_t parity) {
            return !__any_sync(0xffffffffu, !mbar_wait_bounded(bar, parity));
        };
        auto load_keys = [&](int st) {
            const int slot = ki % kRing;
            if (ki >= kRing && !wait_all(k_empty + 8 * slot, ((ki / kRing) - 1) & 1)) return false;
            const int pt = (s0 + st) * kMwTiles + lane;
            int page = -1;
            if (lane < kMwTiles && pt * kPage < L) page = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + pt);
            const bool ok = page >= 0 && page < p.num_pages;  // (other cells are not added to)
            const uint32_t cnt = __popc(__ballot_sync(0xffffffffu, ok));
            if (lane == 0) mbar_expect_tx(k_full + 8 * slot, cnt * kTileBytes);
            __syncwarp();
            if (ok) tma_load_3d(k_s + slot * kMwKBytes + lane * kTileBytes, &tmk, 0, 0, page * p.Hkv + g, k_full + 8 * slot, policy);
            ++ki;
            return true;
        };
        for (int st = 0; many && st < ns; ++st) load_keys(st);  // (no more than the ring holds)
        for (int qb = 0; qb < nqb && !failed; ++qb) {
            if (!sees_run(qb)) continue;
            const int slot = qi % kQSlots;
            if (qi >= kQSlots && !wait_all(q_empty + 8 * slot, ((qi / kQSlots) - 1) & 1)) {
                failed = true;
                break;
            }
            if (lane == 0) {
                mbar_expect_tx(q_full + 8 * slot, Lay::kQBytes + N * 4);
                tma_load_3d_plain(q_s + slot * Lay::kQBytes, &tmq, 0, g * p.G, b * p.T + qb * N / p.G, q_full + 8 * slot);
                bulk_load(smem_addr(s_lse + slot * N), p.nlse + bg * p.lse_ld + qb * N, N * 4, q_full + 8 * slot);
            }
            ++qi;
            __syncwarp();
            for (int st = 0; !many && st < ns; ++st)
                if (sees_stage(qb, st) && !load_keys(st)) {
                    failed = true;
                    break;
                }
        }
        // nothing may still be landing when the CTA leaves
        for (int j = max(0, ki - kRing); j < ki; ++j) wait_all(k_full + 8 * (j % kRing), (j / kRing) & 1);
        for (int j = max(0, qi - kQSlots); j < qi; ++j) wait_all(q_full + 8 * (j % kQSlots), (j / kQSlots) & 1);
    } else if (warp == 9) {
        // ---- MMA issue
        if (lane == 0) {
            const uint32_t idesc = umma_idesc_bf16(kMwKeys, N, false);
            int it = 0, ki = 0, qi = 0;
            for (int qb = 0; qb < nqb && !failed; ++qb) {
                if (!sees_run(qb)) continue;
                const int qs = qi % kQSlots;
                if (!mbar_wait_bounded(q_full + 8 * qs, (qi / kQSlots) & 1)) {
                    failed = true;
                    break;
                }
                for (int st = 0; st < ns; ++st) {
                    if (!sees_stage(qb, st)) continue;
                    const int slot = many ? st : ki % kRing, buf = it & 1;
                    if (!mbar_wait_bounded(k_full + 8 * slot, many ? 0u : (ki / kRing) & 1) ||
                        (it >= 2 && !mbar_wait_bounded(t_empty + 8 * buf, ((it >> 1) - 1) & 1))) {
                        failed = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t ka = k_s + slot * kMwKBytes, qa = q_s + qs * Lay::kQBytes;
#pragma unroll
                    for (int kk = 0; kk < kD / 16; ++kk)
                        umma_bf16_ss(tm + buf * N, umma_sdesc(ka + 32 * kk, 16, 1024), umma_sdesc(qa + 32 * kk, 16, 1024),
                                     idesc, kk > 0);
                    umma_commit(t_full + 8 * buf);
                    if (!many) umma_commit(k_empty + 8 * slot);
                    ++it;
                    ++ki;
                }
                umma_commit(q_empty + 8 * qs);
                ++qi;
            }
            umma_commit(drain);  // completes when every product issued above has
        }
    } else {
        // ---- exponentials and sums: key 32 (warp % 4) + lane of each stage, half warp / 4 of the columns
        const int w = warp & 3, half = warp >> 2;
        const uint32_t lanes = static_cast<uint32_t>(32 * w) << 16;
        int it = 0, qi = 0;
        for (int qb = 0; qb < nqb && !failed; ++qb) {
            if (!sees_run(qb)) continue;
            const int qs = qi % kQSlots;
            if (__any_sync(0xffffffffu, !mbar_wait_bounded(q_full + 8 * qs, (qi / kQSlots) & 1))) {
                failed = true;
                break;
            }
            const float *nlse = s_lse + qs * N + half * kHalf;
            const int r0 = qb * N + half * kHalf;  // the rows of this warp's columns
            for (int st = 0; st < ns; ++st) {
                if (!sees_stage(qb, st)) continue;
                const int buf = it & 1;
                if (__any_sync(0xffffffffu, !mbar_wait_bounded(t_full + 8 * buf, (it >> 1) & 1))) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                ++it;
                // rows that see key j: t >= j - base, t < n, t < j - base + W
                const int j = (s0 + st) * kMwKeys + 32 * w + lane;
                const int t_lo = max(0, j - base), t_hi = W > 0 ? min(n, j - base + W) : n;
                const int lo = t_lo * p.G - r0, hi = j < L ? max(t_lo, t_hi) * p.G - r0 : lo;
                const bool all = __all_sync(0xffffffffu, lo <= 0 && hi >= kHalf);
                const bool any = __any_sync(0xffffffffu, lo < kHalf && hi > 0 && lo < hi);
                const uint32_t ta = tm + lanes + buf * N + half * kHalf;
                float sum = 0.f;
                if (any) {
                    uint32_t v[2][CH];
                    if constexpr (CH == 32) tmem_ld32(ta, v[0]);
                    else tmem_ld16(ta, v[0]);
#pragma unroll
                    for (int c = 0; c < kHalf / CH; ++c) {
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < CH; ++i) asm volatile("" : "+r"(v[c & 1][i]));  // (not used before the wait)
                        if constexpr (CH == 32)
                            if (c + 1 < kHalf / CH) tmem_ld32(ta + 32 * (c + 1), v[(c + 1) & 1]);
                        sum += all ? sum_columns<CH, false>(v[c & 1], nlse + CH * c, p.scale_log2, 0, CH)
                                   : sum_columns<CH, true>(v[c & 1], nlse + CH * c, p.scale_log2, lo - CH * c, hi - CH * c);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(t_empty + 8 * buf);
                const int at = (st * 2 + half) * kMwKeys + 32 * w + lane;
                if (many) {  // compensated: .x the sum, .y what its additions have lost
                    float2 a = reinterpret_cast<float2 *>(s_acc)[at];
                    const float y = sum - a.y, t = a.x + y;
                    a.y = (t - a.x) - y;
                    a.x = t;
                    reinterpret_cast<float2 *>(s_acc)[at] = a;
                } else {
                    s_acc[at] = sum;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(q_empty + 8 * qs);
            ++qi;
        }
    }
    if (failed) {
        flag_status(DA_STATUS_TIMEOUT);
        s_failed = 1;
    }

    // ---- every product done before TMEM is released, every sum before it is added
    if (tid == 9 * 32) mbar_wait_bounded(drain, 0);
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(static_cast<uint32_t>(2 * N)));
    }
    if (s_failed) return;
    for (int i = tid; i < ns * kMwKeys; i += kMwThreads) {
        const int st = i / kMwKeys, j = s0 * kMwKeys + i;
        if (j >= L || j < lo0) continue;
        const int page = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + j / kPage);
        if (page < 0 || page >= p.num_pages) continue;
        const int at = st * 2 * kMwKeys + i % kMwKeys;
        float sum;
        if (many) {
            const float2 a = reinterpret_cast<const float2 *>(s_acc)[at], c = reinterpret_cast<const float2 *>(s_acc)[at + kMwKeys];
            sum = (a.x + c.x) - (a.y + c.y);
        } else {
            sum = s_acc[at] + s_acc[at + kMwKeys];
        }
        float *dst = p.weights + (static_cast<size_t>(page) * p.Hkv + g) * kPage + j % kPage;
        if (p.assign_new && j >= base)
            *dst = sum;
        else
            atomicAdd(dst, sum);
    }
}
