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
// cores (the tcgen05 kernels), since T times as many would cost more to write and read than
// the keys cost to read.

struct WeightParams {
    float *weights;                  // [num_pages][Hkv][16]
    const int *block_table, *seq_lens, *q_lens;
    const float *nlse;               // [B * Hkv][lse_ld]
    int lse_ld;
    float *scores;                   // one token: [unit][16][G]
    float scale_log2;
    int B, Hkv, G, T, window, max_pages, num_pages, max_seq_len;
    int assign_new;                  // the call appended its new tokens
    int run;                         // several tokens, streamed keys: 128-key stages per CTA
};

// ------------------------------------------------------------------ one token per sequence
// Warps take equal contiguous shares of the call's units (16-token tiles in the attention
// kernel's order), one (sequence, KV head) after another with its denominators in registers: one
// token per lane, two tiles per pass, several passes' scores in flight.
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
    constexpr int kPasses = G > 8 ? 1 : G > 4 ? 3 : 4;  // passes in flight (64 registers)
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
    // every CTA of this grid is resident: the next kernel may set itself up as they leave
    if (tid == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    for (int u = ua; u < ue;) {
        const int b = find_seq(s_pre, B, u);
        const int tiles = (s_pre[b + 1] - s_pre[b]) / Hkv, r = u - s_pre[b];
        const int g = r / tiles, t0 = r - g * tiles;
        const int L = s_len[b], lo = (p.window > 0 && L > p.window) ? L - p.window : 0;
        const int pt = lo / kPage + t0, cnt = min(32, min(tiles - t0, ue - u));  // tiles of this batch
        float nl[G];
        load_floats(nl, p.nlse + (static_cast<size_t>(b) * Hkv + g) * G);
        int pages = -1;                                    // lane l: page of tile l
        if (lane < cnt) {
            pages = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + pt + lane);
            if (pages >= p.num_pages) pages = -1;
        }
        const float *sc = p.scores + static_cast<size_t>(u) * (kPage * G) + lane * G;
        for (int i = 0; i < cnt; i += 2 * kPasses) {
            float s[kPasses][G];
#pragma unroll
            for (int k = 0; k < kPasses; ++k)  // (not behind the page: that load is under way too)
                if (i + 2 * k + (lane >> 4) < cnt) load_floats(s[k], sc + (i + 2 * k) * (kPage * G));
#pragma unroll
            for (int k = 0; k < kPasses; ++k) {
                const int tile = i + 2 * k + (lane >> 4), j = (pt + tile) * kPage + (lane & 15);
                const int page = __shfl_sync(0xffffffffu, pages, tile & 31);
                if (tile >= cnt || j < lo || j >= L || page < 0) continue;
                float sum = 0.f;
#pragma unroll
                for (int h = 0; h < G; ++h) sum += fast_exp2(s[k][h] + nl[h]);
                float *dst = p.weights + (static_cast<size_t>(page) * Hkv + g) * kPage + (lane & 15);
                if (p.assign_new && j == L - 1)
                    *dst = sum;
                else
                    atomicAdd(dst, sum);
            }
        }
        // The scores are read once: their lines leave L2 without being written to memory (whole lines
        // of this warp's own tiles; at G = 1 two tiles share one, and a tile's scores are 64 bytes
        // beside 4096 of keys and values: 64 sequences of 1000 to 8192 tokens 104.6 us without the
        // weights, 117.4 with them, 104.8 and 116.7 at G = 2, where the lines are dropped).
        __syncwarp();
        if constexpr (G >= 2)
            for (int i = lane; i < cnt * (G / 2); i += 32)
                asm volatile("discard.global.L2 [%0], 128;" ::"l"(p.scores + static_cast<size_t>(u) * (kPage * G) + 32 * i) : "memory");
        u += cnt;
    }
}

// ------------------------------------------------------------------ several tokens per sequence
// S^T = K Q^T on tcgen05 puts 128 keys on the TMEM lanes (M) and N query rows on the columns, so a
// key's sum over the rows is a sum along a thread's own columns: no shuffles, and the
// denominators are the same for every lane (one broadcast shared-memory read per four columns).
// Two kernels, for what stays in shared memory and what streams past it:
//   stream_keys_weights_kernel<N>      up to 256 query rows per (sequence, KV head): the rows stay
//                                      (N = 32, 64, 128 or 256), 128-key stages stream through a ring
//   stream_rows_weights_kernel<TILES>  more: 128 or 256 keys stay, blocks of 128 query rows stream
// Roles: groups of four warps (128 TMEM lanes each, a share of the columns) form exponentials and
// sums from two TMEM buffers; one warp issues the TMA copies, one thread the products. Keys and
// rows that cannot see each other (causal mask, window) are skipped by every role alike.
constexpr int kMwKeys = 128;
constexpr int kMwTiles = kMwKeys / kPage;
constexpr int kMwKBytes = kMwKeys * kD * 2;  // 16 KiB of keys
constexpr int kMwMaxRows = 256;              // query rows that stay, at most
constexpr int kMwRowBlock = 128;             // query rows per streamed block
constexpr int kMwMaxRun = 16;                // key stages per CTA at most

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

// What a CTA works on: sequence counts and its first key.
struct MwKeys {
    int L, n, base, lo0;
    bool ok;
};
__device__ __forceinline__ MwKeys mw_keys(const WeightParams &p, int b) {
    MwKeys k;
    k.L = __ldg(p.seq_lens + b);
    k.n = p.q_lens != nullptr ? __ldg(p.q_lens + b) : p.T;
    // counts out of range were flagged by the attention
    k.ok = k.L > 0 && k.L <= p.max_seq_len && k.L <= p.max_pages * kPage && k.n > 0 && k.n <= p.T && k.n <= k.L;
    k.base = k.L - k.n;
    k.lo0 = p.window > 0 ? max(0, k.base - p.window + 1) : 0;
    return k;
}

// Query rows [lo, hi) that see key j: tokens t >= j - base, t < n, t < j - base + W.
__device__ __forceinline__ int2 rows_of_key(const WeightParams &p, const MwKeys &k, int j) {
    const int lo = max(0, j - k.base);
    const int hi = j < k.L ? (p.window > 0 ? max(lo, min(k.n, j - k.base + p.window)) : k.n) : lo;
    return make_int2(lo * p.G, hi * p.G);
}

// The key tiles from position `first` on (lane u < tiles: tile u) into dst, counted on bar. Tiles past
// the end and of pages outside the pool are left out: the sums of their keys are not used.
__device__ __forceinline__ void mw_load_keys(const WeightParams &p, const CUtensorMap *tmk, int b, int g, int L, int first,
                                             int tiles, uint32_t dst, uint32_t bar, uint64_t policy, int lane) {
    const int pt = first / kPage + lane;
    int page = -1;
    if (lane < tiles && pt * kPage < L) page = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + pt);
    const bool ok = page >= 0 && page < p.num_pages;
    const uint32_t cnt = __popc(__ballot_sync(0xffffffffu, ok));
    if (lane == 0) mbar_expect_tx(bar, cnt * kTileBytes);
    __syncwarp();
    if (ok) tma_load_3d(dst + lane * kTileBytes, tmk, 0, 0, page * p.Hkv + g, bar, policy);
}

// Sums of `keys` keys from position `first` on to their cells.
template <typename Sum>
__device__ __forceinline__ void mw_add(const WeightParams &p, const MwKeys &k, int b, int g, int first, int keys, Sum sum) {
    for (int i = threadIdx.x; i < keys; i += blockDim.x) {
        const int j = first + i;
        if (j >= k.L || j < k.lo0) continue;
        const int page = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + j / kPage);
        if (page < 0 || page >= p.num_pages) continue;
        float *dst = p.weights + (static_cast<size_t>(page) * p.Hkv + g) * kPage + j % kPage;
        if (p.assign_new && j >= k.base)
            *dst = sum(i);
        else
            atomicAdd(dst, sum(i));
    }
}

// Sum over COLS columns from TMEM column ta on, 32 (or 16) at a time, the next load under way while one
// is summed. MASK: only the columns [lo, hi).
template <int COLS, bool MASK>
__device__ __forceinline__ float sum_tmem(uint32_t ta, const float *nlse, float scale, int lo, int hi) {
    constexpr int CH = COLS < 32 ? 16 : 32;
    uint32_t v[2][CH];
    float sum = 0.f;
    if constexpr (CH == 32) tmem_ld32(ta, v[0]);
    else tmem_ld16(ta, v[0]);
#pragma unroll
    for (int c = 0; c < COLS / CH; ++c) {
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < CH; ++i) asm volatile("" : "+r"(v[c & 1][i]));  // (not used before the wait)
        if constexpr (CH == 32)
            if (c + 1 < COLS / CH) tmem_ld32(ta + 32 * (c + 1), v[(c + 1) & 1]);
        sum += sum_columns<CH, MASK>(v[c & 1], nlse + CH * c, scale, lo - CH * c, hi - CH * c);
    }
    return sum;
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    return !__any_sync(0xffffffffu, !mbar_wait_bounded(bar, parity));
}

template <int N>
struct SkLayout {
    static constexpr int kEpi = N == kMwMaxRows ? 16 : 8;      // warps that sum
    static constexpr int kParts = kEpi / 4;                    // shares of the columns
    static constexpr int kThreads = (kEpi + 2) * 32;
    // resident per SM (N = 32: 4 tokens x 32 sequences 122 us with three CTAs of three stages, 128 with
    // two of four)
    static constexpr int kCtas = N == kMwMaxRows ? 1 : N == 32 ? 3 : 2;
    static constexpr int kRing = N == kMwMaxRows ? 8 : N == 32 ? 3 : 4;
    static constexpr int k = N * kD * 2;
    static constexpr int lse = k + kRing * kMwKBytes;
    static constexpr int acc = lse + N * 4;
    static constexpr int bars = acc + kMwMaxRun * kParts * kMwKeys * 4;
    static constexpr int bytes = 1024 + bars + (2 * kRing + 6) * 8;  // with the slack to align the base
    static_assert(k % 1024 == 0 && acc % 16 == 0 && bars % 8 == 0, "alignment");
    static_assert(kCtas * (bytes + 1024) <= 233472, "shared memory of the CTAs on one SM");
};

// One CTA per (sequence, KV head, run of p.run key stages).
template <int N>
__global__ void __launch_bounds__(SkLayout<N>::kThreads, SkLayout<N>::kCtas)
    stream_keys_weights_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmq,
                               const WeightParams p) {
    using Lay = SkLayout<N>;
    constexpr int kRing = Lay::kRing, kEpi = Lay::kEpi, kCols = N / Lay::kParts;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t q_s = smem_addr(smem), k_s = q_s + Lay::k;
    float *const s_lse = reinterpret_cast<float *>(smem + Lay::lse);
    float *const s_acc = reinterpret_cast<float *>(smem + Lay::acc);
    const uint32_t k_full = smem_addr(smem + Lay::bars), k_empty = k_full + 8 * kRing;
    const uint32_t q_full = k_empty + 8 * kRing, t_full = q_full + 8, t_empty = t_full + 16, drain = t_empty + 16;
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
        mbar_init(q_full, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(t_full + 8 * s, 1);
            mbar_init(t_empty + 8 * s, kEpi);
        }
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s_failed = 0;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const MwKeys k = mw_keys(p, b);
    if (!k.ok) return;
    const int s0 = k.lo0 / kMwKeys + blockIdx.x * p.run;  // first stage: positions 128 s0 on
    const int ns = min(p.run, (k.L - 1) / kMwKeys - s0 + 1);
    if (ns <= 0) return;
    if (warp == kEpi + 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)),
                     "r"(static_cast<uint32_t>(2 * N)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tmem;

    bool failed = false;
    if (warp == kEpi) {
        // ---- TMA
        const uint64_t policy = evict_first_policy();
        if (lane == 0) {
            mbar_expect_tx(q_full, N * kD * 2 + N * 4);
            tma_load_3d_plain(q_s, &tmq, 0, g * p.G, b * p.T, q_full);
            bulk_load(smem_addr(s_lse), p.nlse + (static_cast<size_t>(b) * p.Hkv + g) * p.lse_ld, N * 4, q_full);
        }
        __syncwarp();
        int st = 0;
        for (; st < ns; ++st) {
            const int slot = st % kRing;
            if (st >= kRing && !warp_wait(k_empty + 8 * slot, ((st / kRing) - 1) & 1)) {
                failed = true;
                break;
            }
            mw_load_keys(p, &tmk, b, g, k.L, (s0 + st) * kMwKeys, kMwTiles, k_s + slot * kMwKBytes, k_full + 8 * slot, policy, lane);
        }
        // nothing may still be landing when the CTA leaves
        for (int j = max(0, st - kRing); j < st; ++j) warp_wait(k_full + 8 * (j % kRing), (j / kRing) & 1);
        warp_wait(q_full, 0);
    } else if (warp == kEpi + 1) {
        // ---- products
        if (lane == 0) {
            const uint32_t idesc = umma_idesc_bf16(kMwKeys, N, false);
            // (a stage or a step along the contraction only moves a descriptor's start address)
            const uint64_t dk = umma_sdesc(k_s, 16, 1024), dq = umma_sdesc(q_s, 16, 1024);
            if (!mbar_wait_bounded(q_full, 0)) failed = true;
            for (int st = 0; st < ns && !failed; ++st) {
                const int slot = st % kRing, buf = st & 1;
                if (!mbar_wait_bounded(k_full + 8 * slot, (st / kRing) & 1) ||
                    (st >= 2 && !mbar_wait_bounded(t_empty + 8 * buf, ((st >> 1) - 1) & 1))) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                const uint64_t dks = dk + slot * (kMwKBytes / 16);
#pragma unroll
                for (int kk = 0; kk < kD / 16; ++kk) umma_bf16_ss(tm + buf * N, dks + 2 * kk, dq + 2 * kk, idesc, kk > 0);
                umma_commit(t_full + 8 * buf);
                umma_commit(k_empty + 8 * slot);
            }
            umma_commit(drain);  // completes when every product issued above has
        }
    } else {
        // ---- exponentials and sums: key 32 (warp % 4) + lane of each stage, share warp / 4 of the columns
        const int w = warp & 3, c0 = (warp >> 2) * kCols;
        const uint32_t lanes = static_cast<uint32_t>(32 * w) << 16;
        if (!warp_wait(q_full, 0)) failed = true;
        for (int st = 0; st < ns && !failed; ++st) {
            const int buf = st & 1;
            if (!warp_wait(t_full + 8 * buf, (st >> 1) & 1)) {
                failed = true;
                break;
            }
            tc_fence_after();
            const int2 rows = rows_of_key(p, k, (s0 + st) * kMwKeys + 32 * w + lane);
            const int lo = rows.x - c0, hi = rows.y - c0;
            const uint32_t ta = tm + lanes + buf * N + c0;
            float sum = 0.f;
            if (__all_sync(0xffffffffu, lo <= 0 && hi >= kCols))
                sum = sum_tmem<kCols, false>(ta, s_lse + c0, p.scale_log2, 0, kCols);
            else if (__any_sync(0xffffffffu, lo < kCols && hi > 0 && lo < hi))
                sum = sum_tmem<kCols, true>(ta, s_lse + c0, p.scale_log2, lo, hi);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(t_empty + 8 * buf);
            s_acc[(st * Lay::kParts + (warp >> 2)) * kMwKeys + 32 * w + lane] = sum;
        }
    }
    if (failed) {
        flag_status(DA_STATUS_TIMEOUT);
        s_failed = 1;
    }

    // ---- every product done before TMEM is released, every sum made before it is added
    if (tid == (kEpi + 1) * 32) mbar_wait_bounded(drain, 0);
    tc_fence_before();
    __syncthreads();
    if (warp == kEpi + 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(static_cast<uint32_t>(2 * N)));
    }
    if (s_failed) return;
    mw_add(p, k, b, g, s0 * kMwKeys, ns * kMwKeys, [&](int i) {
        const float *a = s_acc + (i / kMwKeys) * Lay::kParts * kMwKeys + i % kMwKeys;
        float sum = a[0];
#pragma unroll
        for (int q = 1; q < Lay::kParts; ++q) sum += a[q * kMwKeys];
        return sum;
    });
}

template <int TILES>
struct SrLayout {
    static constexpr int kEpi = 8 * TILES;                      // two groups of four warps per 128 keys
    static constexpr int kThreads = (kEpi + 2) * 32;
    static constexpr int kCtas = TILES == 2 ? 1 : 2;            // resident per SM
    static constexpr int kSlots = TILES == 2 ? 6 : 3;
    static constexpr int kQBytes = kMwRowBlock * kD * 2;
    static constexpr int k = kSlots * kQBytes;
    static constexpr int lse = k + TILES * kMwKBytes;
    static constexpr int acc = lse + kSlots * kMwRowBlock * 4;
    static constexpr int bars = acc + TILES * 2 * kMwKeys * 8;
    static constexpr int bytes = 1024 + bars + (2 * kSlots + 6) * 8;  // with the slack to align the base
    static constexpr uint32_t kCols = 2 * TILES * kMwRowBlock;        // TMEM: two buffers
    static_assert(k % 1024 == 0 && acc % 16 == 0 && bars % 8 == 0, "alignment");
    static_assert(kCtas * (bytes + 1024) <= 233472, "shared memory of the CTAs on one SM");
};

// One CTA per (sequence, KV head, 128 TILES keys). A key's sum over thousands of rows is kept as a
// compensated sum over the blocks (terms one after another in 32 bits would lose the last bits).
template <int TILES>
__global__ void __launch_bounds__(SrLayout<TILES>::kThreads, SrLayout<TILES>::kCtas)
    stream_rows_weights_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmq,
                               const WeightParams p) {
    using Lay = SrLayout<TILES>;
    constexpr int kSlots = Lay::kSlots, kEpi = Lay::kEpi, kCols = kMwRowBlock / 2, kKeys = TILES * kMwKeys;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t q_s = smem_addr(smem), k_s = q_s + Lay::k;
    float *const s_lse = reinterpret_cast<float *>(smem + Lay::lse);
    float2 *const s_acc = reinterpret_cast<float2 *>(smem + Lay::acc);
    const uint32_t k_full = smem_addr(smem + Lay::bars), q_full = k_full + 8, q_empty = q_full + 8 * kSlots;
    const uint32_t t_full = q_empty + 8 * kSlots, t_empty = t_full + 16, drain = t_empty + 16;
    __shared__ uint32_t s_tmem;
    __shared__ int s_failed;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // Key blocks are the slowest index: behind a causal mask the first keys are seen by the most rows,
    // so the longest CTAs of every (sequence, KV head) start first.
    const int pairs = p.B * p.Hkv, block = blockIdx.x / pairs, pair = blockIdx.x % pairs;
    const int g = pair % p.Hkv, b = pair / p.Hkv;
    if (tid == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmk)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmq)) : "memory");
        mbar_init(k_full, 1);
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(q_full + 8 * s, 1);
            mbar_init(q_empty + 8 * s, kEpi + 1);  // the products, and the warps that read the denominators
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(t_full + 8 * s, 1);
            mbar_init(t_empty + 8 * s, kEpi);
        }
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s_failed = 0;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const MwKeys k = mw_keys(p, b);
    if (!k.ok) return;
    const int first = k.lo0 / kMwKeys * kMwKeys + block * kKeys;
    if (first >= k.L) return;
    // the blocks of rows that see one of the keys
    const int last = min(first + kKeys, k.L) - 1;
    const int t0 = max(0, first - k.base), t1 = p.window > 0 ? min(k.n - 1, last - k.base + p.window - 1) : k.n - 1;
    const int qb0 = t0 * p.G / kMwRowBlock, nb = max(0, (t1 * p.G + p.G - 1) / kMwRowBlock - qb0 + 1);
    if (warp == kEpi + 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)),
                     "r"(Lay::kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tmem;

    bool failed = false;
    if (warp == kEpi) {
        // ---- TMA
        mw_load_keys(p, &tmk, b, g, k.L, first, TILES * kMwTiles, k_s, k_full, evict_first_policy(), lane);
        int i = 0;
        for (; i < nb; ++i) {
            const int slot = i % kSlots;
            if (i >= kSlots && !warp_wait(q_empty + 8 * slot, ((i / kSlots) - 1) & 1)) {
                failed = true;
                break;
            }
            if (lane == 0) {
                const int r0 = (qb0 + i) * kMwRowBlock;
                mbar_expect_tx(q_full + 8 * slot, Lay::kQBytes + kMwRowBlock * 4);
                tma_load_3d_plain(q_s + slot * Lay::kQBytes, &tmq, 0, g * p.G, b * p.T + r0 / p.G, q_full + 8 * slot);
                bulk_load(smem_addr(s_lse + slot * kMwRowBlock), p.nlse + (static_cast<size_t>(b) * p.Hkv + g) * p.lse_ld + r0,
                          kMwRowBlock * 4, q_full + 8 * slot);
            }
            __syncwarp();
        }
        // nothing may still be landing when the CTA leaves
        warp_wait(k_full, 0);
        for (int j = max(0, i - kSlots); j < i; ++j) warp_wait(q_full + 8 * (j % kSlots), (j / kSlots) & 1);
    } else if (warp == kEpi + 1) {
        // ---- products
        if (lane == 0) {
            const uint32_t idesc = umma_idesc_bf16(kMwKeys, kMwRowBlock, false);
            const uint64_t dk = umma_sdesc(k_s, 16, 1024), dq = umma_sdesc(q_s, 16, 1024);
            if (!mbar_wait_bounded(k_full, 0)) failed = true;
            for (int i = 0; i < nb && !failed; ++i) {
                const int slot = i % kSlots, buf = i & 1;
                if (!mbar_wait_bounded(q_full + 8 * slot, (i / kSlots) & 1) ||
                    (i >= 2 && !mbar_wait_bounded(t_empty + 8 * buf, ((i >> 1) - 1) & 1))) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                const uint64_t dqs = dq + slot * (Lay::kQBytes / 16);
#pragma unroll
                for (int m = 0; m < TILES; ++m)
#pragma unroll
                    for (int kk = 0; kk < kD / 16; ++kk)
                        umma_bf16_ss(tm + (buf * TILES + m) * kMwRowBlock, dk + m * (kMwKBytes / 16) + 2 * kk, dqs + 2 * kk,
                                     idesc, kk > 0);
                umma_commit(t_full + 8 * buf);
                umma_commit(q_empty + 8 * slot);
            }
            umma_commit(drain);  // completes when every product issued above has
        }
    } else {
        // ---- exponentials and sums: one key per thread, half of each block's columns
        const int m = warp >> 3, half = (warp >> 2) & 1, w = warp & 3, c0 = half * kCols;
        const int2 rows = rows_of_key(p, k, first + m * kMwKeys + 32 * w + lane);
        // rows seen by all of the warp's keys, and by any of them
        const int all_lo = __reduce_max_sync(0xffffffffu, rows.x), all_hi = __reduce_min_sync(0xffffffffu, rows.y);
        const int any_lo = __reduce_min_sync(0xffffffffu, rows.x), any_hi = __reduce_max_sync(0xffffffffu, rows.y);
        const uint32_t ta0 = tm + (static_cast<uint32_t>(32 * w) << 16) + m * kMwRowBlock + c0;
        float sum = 0.f, lost = 0.f;  // compensated: what the additions to sum have lost
        for (int i = 0; i < nb; ++i) {
            const int slot = i % kSlots, buf = i & 1;
            // (the denominators came with the rows: their barrier has completed, this wait makes them visible)
            if (!warp_wait(t_full + 8 * buf, (i >> 1) & 1) || !warp_wait(q_full + 8 * slot, (i / kSlots) & 1)) {
                failed = true;
                break;
            }
            tc_fence_after();
            const int r0 = (qb0 + i) * kMwRowBlock + c0;
            const uint32_t ta = ta0 + buf * TILES * kMwRowBlock;
            const float *nlse = s_lse + slot * kMwRowBlock + c0;
            float add = 0.f;
            if (r0 >= all_lo && r0 + kCols <= all_hi)
                add = sum_tmem<kCols, false>(ta, nlse, p.scale_log2, 0, kCols);
            else if (r0 < any_hi && r0 + kCols > any_lo)
                add = sum_tmem<kCols, true>(ta, nlse, p.scale_log2, rows.x - r0, rows.y - r0);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(t_empty + 8 * buf);
                mbar_arrive(q_empty + 8 * slot);
            }
            const float y = add - lost, t = sum + y;
            lost = (t - sum) - y;
            sum = t;
        }
        s_acc[(m * 2 + half) * kMwKeys + 32 * w + lane] = make_float2(sum, lost);
    }
    if (failed) {
        flag_status(DA_STATUS_TIMEOUT);
        s_failed = 1;
    }

    // ---- every product done before TMEM is released, every sum made before it is added
    if (tid == (kEpi + 1) * 32) mbar_wait_bounded(drain, 0);
    tc_fence_before();
    __syncthreads();
    if (warp == kEpi + 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(Lay::kCols));
    }
    if (s_failed) return;
    mw_add(p, k, b, g, first, kKeys, [&](int i) {
        const float2 a = s_acc[i / kMwKeys * 2 * kMwKeys + i % kMwKeys], c = s_acc[(i / kMwKeys * 2 + 1) * kMwKeys + i % kMwKeys];
        return (a.x + c.x) - (a.y + c.y);
    });
}
