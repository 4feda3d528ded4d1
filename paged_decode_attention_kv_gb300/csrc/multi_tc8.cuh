// Several query tokens per sequence over an fp8 cache, on the 5th-generation tensor cores: the
// step of multi_tc_kernel with its keys and values in fp8 blocks. The new tokens were quantised
// into their blocks by the kernel before (kv_append_fp8_kernel), so every key is read from the
// cache: query row (t, h) at position p = L - n + t attends the cached positions lo .. p.
//
// The codes are turned into fp16 operands in shared memory, their token's scale with them. A page
// (16 tokens) has a power of two 2^E for its K scales, 2^F for its V scales, the largest scale below 2^7 times it, and
//     K'_j = fp16(code_j ks_j 2^-E),   V'_j = fp16(code_j fp16(vs_j 2^-F)):
// code times a factor of at most 2^7: 448 x 128 = 57344, nothing to overflow, and a scale of 2^-20 of its page's largest
// still has a factor with all of fp16's bits. K' is rounded once (its factor is carried as two
// fp16 values: an error of the factor would move all of a token's score), V' twice, each time by at most
// fp16's half step 2^-11. A row of zeros, whose scale is 1 by the format whatever the rows around it, counts in
// neither power: it would push small scales' factors below fp16's range, and in V all the other pages'
// probabilities. 2^E goes into the page's score multiplier; 2^F into the exponent of
// its probabilities, so that the output accumulates in one unit:
//     s_j + F = (q K'_j) (scale log2(e) 2^E) + F,   P_j = fp16(2^(s_j + F - R + 7)),
//     O = sum P_j V'_j = 2^(7-R) sum 2^(s_j) v_j,   l = sum over pages 2^-F sum P_j = 2^(7-R) sum 2^(s_j)
// with R a running reference of s_j + F per row (the next integer, moved only when exceeded by more
// than 2^8, as in multi_tc_kernel): the probabilities stay below 2^15, and fp16 holds them to 2^-12 (to 2^-31 of the
// largest for the smallest ones). Multiplying the scores by their token's scale in the softmax
// instead would be exact, but every factor is then read from shared memory by every row: 4 bytes a
// lane and key, more than the whole softmax takes. Scales below 2^-100 (K) and 2^-60 (V) lose bits; above 2^100 and
// 2^60 an operand may become infinite. V's range is the narrower one because it stands in the exponents of fp32
// probabilities: pages 2^120 apart still count in the same denominators.
//
// The work is cut on the device: a unit is a block of 64 keys of a segment (sequence, KV head, block of
// 128 query rows); a segment costs its units and kT8SegCost more, for its start and end, and every CTA of the grid (two
// per SM) takes the same cost of consecutive units, whatever the lengths. A segment that lies in one CTA is finished
// there; one that is shared leaves fp32 partials (m, l, O per row; two slots per CTA), folded by the CTA that comes last,
// or, where the host sees that a few segments fill the whole grid, by t8_combine_kernel. With a grid of (segment, key
// split) CTAs cut for the longest sequence instead, 64 sequences of 1024 to 8192 tokens took 248 us.
//
// 16 warps stream through the CTA's units without a break between segments:
//   warps 0-3   one query row per thread (TMEM lane = row): the softmax and the finish
//   warps 4-11  two teams of four that take turns: warp u of a team turns tile u of its unit into K' and V'
//   warp 12     issues the MMAs: S_i = Q K'_i^T and O += P_i V'_i (V' as it is stored, transposed:
//               tokens contiguous, so both operands are K-major)
//   warp 13     copies the units' fp8 blocks (2176 bytes each, one bulk copy), lane u tile u
//   warps 14-15 the next segment's query rows as fp16 into the other of two Q buffers, and its place for the row
//               warps (done by the row warps themselves, with their partials' stores a row at a time, 64 sequences x 16
//               tokens took 194 us instead of 173, four prompts 402 instead of 350)
// Two teams because one is a chain of latencies (copy landed, scales' maximum, factors, operands) of about
// 2400 cycles a unit. Registers go where they are needed (setmaxnreg): 64 a thread at launch, then 88 for
// the rows, 56 for the others, 4 x 64 in all.
// The softmax takes the probabilities with the reference it has, and looks for a larger one only if a
// tile's sum shows that one may have left fp16's range: the scores then still stand in TMEM (P has its own columns)
// and are taken again. The maxima of every unit cost 40 of its 230 instructions. A segment's first unit is tried with
// the last segment's reference and taken again if its probabilities are too small for fp16, too (without: four prompts
// 297 us instead of 262). It works a tile (16 keys) at a time and fetches the next one's scores meanwhile: 32 keys at a
// time, one after the other, took 173 us for 64 x 16 tokens instead of 168.
//
// What bounds it: the ring S issued -> scores -> probabilities -> P stored -> PV issued, and behind it the stage that PV
// frees and the teams' next operands: about 2000 cycles a unit with two CTAs on an SM, 1400 of them the rows' work. The SM
// issues 52% of the time (2470 instructions a unit: rows 1090, teams 700, waits, copies and MMAs the rest); the tensor
// cores work 21% of it, the exponentials' unit 256 cycles a unit. A segment's start and end are worth about 4 units.
// 64 sequences of 1024 to 8192 tokens, 16 tokens each: 148 us (2.2 TB/s, 503 TFLOP/s); 512 tokens behind 7680: 124 us
// (537 TFLOP/s); four prompts of 1201 to 2048: 236 us; 16 tokens behind 65536 of 19 sequences: 635 TFLOP/s; G = 8, 64
// query heads throughout (the look for rows of zeros: 1 to 2% of it). Tried, without a gain or slower: four stages, more raw
// units, S and PV by two warps, S_i before PV_{i-2} (the stage comes free later: 171 us instead of 156), outputs in whole
// lines through shared memory (the query buffer is then held to the segment's end: 297 us instead of 268 for the prompts),
// registers 96 / 56 / 48, 88 / 48 / 72, 80 / 56 / 64, 104 / 48 / 56, all 64 scores in registers (they spill).
constexpr int kT8Rows = 128, kT8Keys = 64, kT8Tiles = kT8Keys / kPage;
constexpr int kT8Stages = 3;  // blocks of K' and V'
constexpr int kT8Raw = 2;     // units of fp8 blocks in flight
// An even number: every raw block is always the same team's. With three, a team could wait for its unit's
// parity on a barrier whose last unit, the other team's, had not landed yet, and take the phase before for its own.
// (The stages are safe with any number: a team's unit i - 2 has seen PV_{i-5} done, so that the phase before the one
// it waits for, PV_{i-6}'s, is over.)
static_assert(kT8Raw % 2 == 0, "a raw block belongs to one team");
constexpr int kT8HalfBytes = kT8Keys * kD * 2;  // 8 KiB of K' (or V')
constexpr int kT8StageBytes = 2 * kT8HalfBytes;
constexpr int kT8QBytes = kT8Rows * kD * 2;
constexpr int kT8RawBytes = kT8Tiles * kT8Raw * kBlk8Bytes;
constexpr int kT8Bars = 2 * kT8Raw + 2 * kT8Stages + 5 * 2 + 1;
constexpr int kT8Smem = 1024 + 2 * kT8QBytes + kT8Stages * kT8StageBytes + kT8RawBytes + kT8Stages * kT8Tiles * 16 + kT8Bars * 8;
constexpr int kT8Warps = 16, kT8Threads = kT8Warps * 32, kT8CtasPerSm = 2;
static_assert(kT8CtasPerSm * (kT8Smem + 1024 + 1024) <= 233472, "two CTAs' shared memory on one SM");
static_assert((kMaxBatch + 1) * 12 <= kT8Stages * kT8StageBytes, "the prefixes of costs and segments fit the stages");
constexpr uint32_t kT8TmemCols = 256, kT8ColS = 0, kT8ColO = 128, kT8ColP = 192;  // S and P: two buffers each
constexpr float kT8Shift = 7.f, kT8TileMax = 32768.f;  // log2 of the probabilities' unit; the most a tile's may add up to
constexpr float kT8Ahead = 8.f;  // log2 of how far a score may lie above the reference (none alone passes kT8TileMax then)
// The power of two above a page's largest scale, at most (and at least, negated): scales up to 2^100, 2^60; and log2 of
// what the factors may rise to.
constexpr int kT8MaxE = 101, kT8MaxF = 61, kT8Room = 7;
constexpr int kT8Counters = 4 * kT8CtasPerSm * kMaxSms;  // arrivals at a shared segment: one per row warp, at its first CTA
// What a segment's start and end cost, in units. A prompt's first row blocks see few keys, and CTAs that took as many
// units as the others had several times their segments. With 3 / 4 / 5 / 6, four prompts took 237 / 230 / 232 / 235 us,
// 64 sequences x 16 tokens 150 / 148 / 150 / 149, slots behind a window 75 each, a 512-token chunk 123 each; with 0
// instead of 6, when a start cost more than now, 333 instead of 268, 165 instead of 156 and 82 instead of 78.
constexpr int kT8SegCost = 4;
// A CTA's share at least, where there is so little: with 4 / 8 / 10, 36 short slots (9 to 300 tokens) took 35 / 30 / 32 us,
// 16 tokens behind 1024 30 / 31 / 28, behind 4096 28 / 27 / 28, four prompts of 100 to 300 42 each.
constexpr int kT8MinCost = 8;
constexpr size_t kT8SlotFloats = static_cast<size_t>(kT8Rows) * (2 + kD);

__host__ __device__ constexpr uint32_t umma_idesc_f16(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// A sequence's counts (n = 0: nothing to do), and its row blocks with queries: the first `blocks`.
struct T8Seq {
    int L, n, blocks;
    bool bad;
};
__device__ __forceinline__ T8Seq t8_seq(const MultiParams &p, int b) {
    T8Seq s;
    s.L = __ldg(p.seq_lens + b);
    s.n = p.q_lens != nullptr ? __ldg(p.q_lens + b) : p.T;
    s.bad = s.L < 0 || s.n < 0 || s.n > p.T || (s.L > 0 && s.n > s.L) || s.L > p.max_seq_len ||
            s.L > static_cast<long long>(p.max_pages) * kPage;
    if (s.bad || s.L == 0) s.L = s.n = 0;
    s.blocks = (s.n * p.G + kT8Rows - 1) / kT8Rows;
    return s;
}
// The keys [lo, end) of row block rb of a sequence, its first tile and its units.
struct T8Keys {
    int lo, end, pt_lo, ntiles, units;
};
__device__ __forceinline__ T8Keys t8_keys(const MultiParams &p, const T8Seq &s, int rb) {
    T8Keys k;
    const int base = s.L - s.n;
    const int t0 = rb * kT8Rows / p.G, t1 = min(s.n - 1, (rb * kT8Rows + kT8Rows - 1) / p.G);
    k.lo = p.window > 0 ? max(0, base + t0 - p.window + 1) : 0;
    k.end = base + t1 + 1;
    k.pt_lo = k.lo / kPage;
    k.ntiles = (k.end - 1) / kPage - k.pt_lo + 1;
    k.units = (k.ntiles + kT8Tiles - 1) / kT8Tiles;
    return k;
}
// The cost of a row block.
__device__ __forceinline__ int t8_cost(const MultiParams &p, const T8Seq &s, int rb) { return kT8SegCost + t8_keys(p, s, rb).units; }

// a[1 .. B] added up by a warp, from a[0] = 0.
template <typename N>
__device__ __forceinline__ void t8_scan(N *a, int B, int lane) {
    N run = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
        const int b = b0 + lane;
        N x = b < B ? a[b + 1] : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const N y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        if (b < B) a[b + 1] = run + x;
        run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) a[0] = 0;
}

// Exclusive prefixes over the sequences (all KV heads) of their cost into pre[0 .. B] and of their segments into segs
// (null: not wanted), by all threads of the CTA.
__device__ __forceinline__ void t8_prefix(const MultiParams &p, long long *pre, int *segs, int warp, int nwarps, int lane) {
    const int tid = warp * 32 + lane;
    if (p.row_blocks <= 4) {  // a thread per sequence
        for (int b = tid; b < p.B; b += nwarps * 32) {
            const T8Seq s = t8_seq(p, b);
            long long sum = 0;
            for (int rb = 0; rb < s.blocks; ++rb) sum += t8_cost(p, s, rb);
            pre[b + 1] = sum * p.Hkv;
            if (segs != nullptr) segs[b + 1] = s.blocks * p.Hkv;
        }
    } else {
        for (int b = warp; b < p.B; b += nwarps) {
            const T8Seq s = t8_seq(p, b);
            long long sum = 0;
            for (int rb = lane; rb < s.blocks; rb += 32) sum += t8_cost(p, s, rb);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if (lane == 0) {
                pre[b + 1] = sum * p.Hkv;
                if (segs != nullptr) segs[b + 1] = s.blocks * p.Hkv;
            }
        }
    }
    __syncthreads();
    if (warp == 0) t8_scan(pre, p.B, lane);
    if (warp == 1 && segs != nullptr) t8_scan(segs, p.B, lane);
    __syncthreads();
}

// CTA c of nc takes the places [c U / nc, (c + 1) U / nc) of all U; the CTA that holds place x.
__device__ __forceinline__ long long t8_first(long long U, int nc, int c) { return c * U / nc; }
__device__ __forceinline__ int t8_owner(long long U, int nc, long long x) { return static_cast<int>(((x + 1) * nc - 1) / U); }
__device__ __forceinline__ int t8_ctas(long long U, int grid) {
    return static_cast<int>(max(1ll, min(static_cast<long long>(grid), (U + kT8MinCost - 1) / kT8MinCost)));
}

// The segment that place x lies in, found by a warp.
struct T8At {
    int b, g, rb, units;
    long long begin, before;  // the place of its first unit; the units of all segments before it
};
__device__ __forceinline__ T8At t8_at(const MultiParams &p, const long long *pre, const int *segs, long long x, int lane) {
    int lo = 0, hi = p.B - 1;  // the last sequence that starts at or before it
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    const T8Seq s = t8_seq(p, lo);
    const long long per = (pre[lo + 1] - pre[lo]) / p.Hkv;
    T8At at;
    at.b = lo;
    at.g = static_cast<int>((x - pre[lo]) / per);
    at.rb = at.units = 0;
    long long start = pre[lo] + at.g * per;
    for (int r0 = 0; r0 < s.blocks; r0 += 32) {  // 32 row blocks at a time
        const int u = r0 + lane < s.blocks ? t8_cost(p, s, r0 + lane) : 0;
        int sum = u;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += y;
        }
        const uint32_t in = __ballot_sync(0xffffffffu, x < start + sum);
        if (in != 0) {
            const int k = __ffs(static_cast<int>(in)) - 1;
            start += __shfl_sync(0xffffffffu, sum - u, k);
            at.rb = r0 + k;
            at.units = __shfl_sync(0xffffffffu, u, k) - kT8SegCost;
            break;
        }
        start += __shfl_sync(0xffffffffu, sum, 31);
    }
    at.begin = start + kT8SegCost;
    at.before = start - static_cast<long long>(kT8SegCost) * (segs[lo] + at.g * s.blocks + at.rb);
    return at;
}

// A walk over a CTA's units, segment by segment: the segment's place and keys, and the units [u0, u1)
// of it that are the CTA's.
struct T8Walk {
    int b, g, rb, u0, u1;
    long long begin, end;  // the place of the segment's first unit, the CTA's last place + 1
    T8Seq seq;
    T8Keys keys;
    __device__ __forceinline__ void cut() { u1 = static_cast<int>(min(static_cast<long long>(keys.units), end - begin)); }
    __device__ __forceinline__ void start(const MultiParams &p, const int4 &at, const long long *range) {
        b = at.x, g = at.y, rb = at.z, u0 = at.w, begin = range[0], end = range[1];
        seq = t8_seq(p, b);
        keys = t8_keys(p, seq, rb);
        cut();
    }
    __device__ __forceinline__ bool next(const MultiParams &p) {  // false: that was the last one
        const long long then = begin + keys.units + kT8SegCost;
        if (then >= end) return false;
        begin = then;
        if (++rb >= seq.blocks) {
            rb = 0;
            if (++g >= p.Hkv) {
                g = 0;
                do seq = t8_seq(p, ++b);
                while (seq.blocks == 0);
            }
        }
        keys = t8_keys(p, seq, rb);
        u0 = 0;
        cut();
        return true;
    }
};

// What the row warps need of a segment, from the warps that load its query rows.
struct T8Seg {
    int b, g, rb, n, base;        // base: position of the first new token
    int pt_lo, u0, u1, units;     // first tile; the CTA's units [u0, u1) of all
    int last;
    long long begin;              // the place of the segment's first unit
};

// Partials of a segment: m [128 rows], l [128 rows], O as [16][128 rows] float4 (so that 32 rows' loads and stores are
// contiguous). Contributor i: the first one's in its CTA's slot k0, the others' in slot 0.
__device__ __forceinline__ const float *t8_slot(const MultiParams &p, int c0, int k0, int i) {
    return p.part + (static_cast<size_t>(c0 + i) * 2 + (i == 0 ? k0 : 0)) * kT8SlotFloats;
}
__device__ __forceinline__ const float4 *t8_acc(const float *slot, int c, int rl) {
    return reinterpret_cast<const float4 *>(slot + 2 * kT8Rows) + c * kT8Rows + rl;
}

// A row's partials folded with the sink by one thread, for the CTA that folds a few of them.
__device__ __noinline__ void t8_fold(const MultiParams &p, int c0, int k0, int count, int rl, int head, bool query, uint4 *out) {
    float M = -INFINITY;
    if (query) {
#pragma unroll 4
        for (int i = 0; i < count; ++i) M = fmaxf(M, __ldcg(t8_slot(p, c0, k0, i) + rl));
    }
    const float sg = query && p.sinks != nullptr ? __ldg(p.sinks + head) * kLog2e : -INFINITY;
    const float Mf = fmaxf(M, sg);
    float d = sg == -INFINITY ? 0.f : exp2f(sg - Mf);
    if (Mf != -INFINITY) {
#pragma unroll 4
        for (int i = 0; i < count; ++i) {
            const float m = __ldcg(t8_slot(p, c0, k0, i) + rl), l = __ldcg(t8_slot(p, c0, k0, i) + kT8Rows + rl);
            d += m == -INFINITY ? 0.f : l * exp2f(m - Mf);
        }
    }
    const float inv = d > 0.f ? 1.f / d : d == d ? 0.f : d;
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
        float4 o[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (Mf != -INFINITY)
            for (int i = 0; i < count; ++i) {
                const float *s = t8_slot(p, c0, k0, i);
                const float m = __ldcg(s + rl), w = m == -INFINITY ? 0.f : exp2f(m - Mf);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float4 x = __ldcg(t8_acc(s, 8 * h + c, rl));
                    if (w == 0.f) continue;  // (no key there: the accumulator was not written)
                    o[c].x += x.x * w, o[c].y += x.y * w, o[c].z += x.z * w, o[c].w += x.w * w;
                }
            }
#pragma unroll
        for (int c = 0; c < 4; ++c)
            out[4 * h + c] = make_uint4(pack_bf16(o[2 * c].x * inv, o[2 * c].y * inv), pack_bf16(o[2 * c].z * inv, o[2 * c].w * inv),
                                        pack_bf16(o[2 * c + 1].x * inv, o[2 * c + 1].y * inv), pack_bf16(o[2 * c + 1].z * inv, o[2 * c + 1].w * inv));
    }
}

// expire: -1, or 8 i + role: the first CTA's warp of that role (0: row warp 0, 1: tile 0 of the team that has unit i, 2:
// copies, 3: MMAs, 4: query rows, first half) gives up at unit i (1, 2) or at segment i, as if its wait there had expired
// (decode_attn_test_expire_wait). Looked at outside the loops over units: looks in them took 7 to 10% of a call.
__global__ void __launch_bounds__(kT8Threads, kT8CtasPerSm)
    multi_tc8_kernel(const MultiParams p, const uint8_t *__restrict__ kv, const int expire) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *sQ = smem;                        // [2][128 rows][128 B], 128-byte swizzle
    uint8_t *sKV = smem + 2 * kT8QBytes;       // [stage][K' block [64 tokens][128 B] | V' block [64 d][128 B]]
    uint8_t *sRaw = sKV + kT8Stages * kT8StageBytes;  // [kT8Raw][tile][2176]
    float4 *s_fac = reinterpret_cast<float4 *>(sRaw + kT8RawBytes);  // [stage][tile]: multiplier, F, 2^-F, bits: the unit is a segment's first
    uint64_t *bars = reinterpret_cast<uint64_t *>(s_fac + kT8Stages * kT8Tiles);
    const uint32_t raw_full = smem_addr(bars), raw_empty = raw_full + 8 * kT8Raw;
    const uint32_t kv_full = raw_empty + 8 * kT8Raw, kv_empty = kv_full + 8 * kT8Stages;
    const uint32_t s_full = kv_empty + 8 * kT8Stages, p_full = s_full + 16, o_done = p_full + 16;
    const uint32_t q_full = o_done + 16, q_free = q_full + 16, drain = q_free + 16;
    __shared__ __align__(16) uint32_t s_vfac[2 * kT8Tiles][kPage / 2];  // V factors of a tile: 16 fp16 values
    // a raw tile's tokens that are keys: [x & 255, x >> 8 & 255), none where there is no page; bit 16: its unit is the
    // segment's first here
    __shared__ int s_keys[kT8Raw][kT8Tiles];
    __shared__ T8Seg s_seg[4];
    __shared__ int4 s_start;
    __shared__ long long s_range[3];  // the place of the first segment's first unit, the CTA's last place + 1, all places
    __shared__ long long s_before[2]; // the units before the CTA's places, and before those after them
    __shared__ uint32_t s_tmem;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    if (tid == 0) {
        for (int s = 0; s < kT8Raw; ++s) {
            mbar_init(raw_full + 8 * s, 1);
            mbar_init(raw_empty + 8 * s, kT8Tiles);
        }
        for (int s = 0; s < kT8Stages; ++s) {
            mbar_init(kv_full + 8 * s, kT8Tiles);
            mbar_init(kv_empty + 8 * s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(s_full + 8 * s, 2);  // the products, and the issuing thread
            mbar_init(p_full + 8 * s, 4);  // the four row warps
            mbar_init(o_done + 8 * s, 1);
            mbar_init(q_full + 8 * s, 2);  // the two warps that load query rows
            mbar_init(q_free + 8 * s, 5);  // the segment's products done, and the row warps past q_full (the products of a
                                           // segment of one unit can be done before the rows have looked)
        }
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)),
                     "r"(kT8TmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    // The kernel before is this call's append, which waited for everything before it and let this one start only
    // then: all but the cache may be read, and the output written, at once. Warp 13, which copies from the cache, waits.

    // ---- the CTA's units; the output rows that have no query: zeros
    long long *pre = reinterpret_cast<long long *>(sKV);
    int *segs = reinterpret_cast<int *>(pre + kMaxBatch + 1);
    t8_prefix(p, pre, segs, warp, kT8Warps, lane);
    const long long U = pre[p.B];
    const int nc = t8_ctas(U, gridDim.x), cta = blockIdx.x;
    if (warp < 2) {
        const long long first = cta < nc ? t8_first(U, nc, cta) : U, end = cta < nc ? t8_first(U, nc, cta + 1) : U;
        const long long x = warp == 0 ? first : end;
        long long before = U - static_cast<long long>(kT8SegCost) * segs[p.B];
        if (x < U) {
            const T8At at = t8_at(p, pre, segs, x, lane);
            const long long u = max(0ll, x - at.begin);  // its units before x
            before = at.before + u;
            if (warp == 0 && lane == 0) {
                s_start = make_int4(at.b, at.g, at.rb, static_cast<int>(u));
                s_range[0] = at.begin;
            }
        }
        if (lane == 0) {
            s_before[warp] = before;
            s_range[1 + warp] = warp == 0 ? end : U;
        }
    }
    for (int i = cta; i < p.B * p.row_blocks; i += gridDim.x) {
        const int b = i / p.row_blocks, rb = i - b * p.row_blocks;
        const T8Seq s = t8_seq(p, b);
        if (s.bad && rb == 0 && tid == 0) flag_status(DA_STATUS_BAD_SEQ_LEN);
        if (rb < s.blocks) continue;
        const int r0 = rb * kT8Rows, rows = min(kT8Rows, p.T * p.G - r0);
        for (int j = tid; j < rows * p.Hkv * (kD / 8); j += kT8Threads) {
            const int c = j & 7, r = r0 + (j >> 3) % rows, g = (j >> 3) / rows, t = r / p.G;
            reinterpret_cast<uint4 *>(p.out + ((static_cast<size_t>(b) * p.T + t) * p.Hq + g * p.G + (r - t * p.G)) * kD)[c] =
                make_uint4(0, 0, 0, 0);
        }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the stages held the prefix
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tmem;
    const int units = static_cast<int>(s_before[1] - s_before[0]);

    auto gives_up = [&](int role, int i) { return expire == 8 * i + role && blockIdx.x == 0; };
    auto units_of = [&](int role) {  // the units that a role goes through: all, or up to where it gives up
        return expire >= 0 && blockIdx.x == 0 && (expire & 7) == role ? min(units, expire >> 3) : units;
    };
    bool failed = false;
    if (warp >= 4 && warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        // ---- operands: tile u of every other unit
        const int u = warp & 3, team = (warp - 4) >> 2;
        unsigned short *const vfac = reinterpret_cast<unsigned short *>(s_vfac[warp - 4]);
        int st = team % kT8Stages, rs = team % kT8Raw;
        uint32_t st_ph = 1, rs_ph = 0;  // (the first round of stages is free)
        const int all = u == 0 ? units_of(1) : units;
        failed = all < units && (all & 1) == team;
        for (int i = team; i < all; i += 2) {
            if (__any_sync(0xffffffffu, !mbar_wait_bounded(raw_full + 8 * rs, rs_ph))) {
                failed = true;
                break;
            }
            const uint8_t *blk = sRaw + (rs * kT8Tiles + u) * kBlk8Bytes;
            const int keys = s_keys[rs][u], key_a = keys & 255, key_e = keys >> 8 & 255;
            float sc = reinterpret_cast<const float *>(blk + kBlk8S)[lane];
            uint4 kc[2], vc[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                kc[h] = reinterpret_cast<const uint4 *>(blk)[lane + 32 * h];
                vc[h] = reinterpret_cast<const uint4 *>(blk + kBlk8V)[lane + 32 * h];
            }
            if ((keys & 0xffff) != kPage << 8) {
                // a token outside the rows' keys may hold anything: its codes and scales are zeros
                auto key = [&](int t) { return t >= key_a && t < key_e; };
                if (!key(lane & 15)) sc = 0.f;
                uint32_t m[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    m[e] = (key(4 * e) ? 0xffu : 0u) | (key(4 * e + 1) ? 0xff00u : 0u) |
                           (key(4 * e + 2) ? 0xff0000u : 0u) | (key(4 * e + 3) ? 0xff000000u : 0u);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!key((lane >> 2) + 8 * h)) kc[h] = make_uint4(0, 0, 0, 0);
                    vc[h] = make_uint4(vc[h].x & m[0], vc[h].y & m[1], vc[h].z & m[2], vc[h].w & m[3]);
                }
            }
            // rows of zeros, looked for where a scale is theirs (K: lanes 0-15, V: 16-31): they have no scale
            if (__any_sync(0xffffffffu, sc == 1.f)) {
                // (four lanes hold a K row, so that a token has four bits of a vote)
                const uint32_t k0 = __ballot_sync(0xffffffffu, ((kc[0].x | kc[0].y | kc[0].z | kc[0].w) & 0x7f7f7f7fu) != 0);
                const uint32_t k1 = __ballot_sync(0xffffffffu, ((kc[1].x | kc[1].y | kc[1].z | kc[1].w) & 0x7f7f7f7fu) != 0);
                uint32_t any = (lane & 8 ? k1 : k0) >> (4 * (lane & 7)) & 15u;
                // (a lane holds two elements of V of all tokens, four to a word)
                const uint32_t w[4] = {vc[0].x | vc[1].x, vc[0].y | vc[1].y, vc[0].z | vc[1].z, vc[0].w | vc[1].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t all = __reduce_or_sync(0xffffffffu, w[e]);
                    if (lane >> 2 == 4 + e) any = all >> (8 * (lane & 3)) & 127u;
                }
                if (any == 0) sc = 0.f;
            }
            // the page's powers of two, and each token's factor
            float top = fabsf(sc);
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const int lim = lane < 16 ? kT8MaxE : kT8MaxF;
            const int ex = max(-lim, min(lim, static_cast<int>(__float_as_uint(top) >> 23) - 126));
            const float down = __uint_as_float(static_cast<uint32_t>(127 + kT8Room - ex) << 23);
            const float fac = sc * down;
            const __half hi = __float2half_rn(fac), lo = __float2half_rn(fac - __half2float(hi));
            const uint32_t packed = static_cast<uint32_t>(__half_as_ushort(hi)) | static_cast<uint32_t>(__half_as_ushort(lo)) << 16;
            if (lane >= 16) vfac[lane - 16] = __half_as_ushort(hi);
            __syncwarp();
            if (lane == 0) mbar_arrive(raw_empty + 8 * rs);  // the raw block has been read
            const uint4 f0 = reinterpret_cast<const uint4 *>(vfac)[0], f1 = reinterpret_cast<const uint4 *>(vfac)[1];
            const uint32_t vf[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
            if (__any_sync(0xffffffffu, !mbar_wait_bounded(kv_empty + 8 * st, st_ph))) {
                failed = true;
                break;
            }
            float *fo = reinterpret_cast<float *>(s_fac + st * kT8Tiles + u);
            if (lane == 0) fo[0] = fmaxf(p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - kT8Room + ex) << 23), 1.1754944e-38f);
            if (lane == 16) {
                fo[1] = static_cast<float>(ex - kT8Room);
                fo[2] = down;
                fo[3] = __int_as_float(keys >> 16);
            }
            uint8_t *sK = sKV + st * kT8StageBytes, *sV = sK + kT8HalfBytes;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                {  // K: token (lane / 4) + 8 h, elements 16 (lane % 4) .. + 15
                    const int t = (lane >> 2) + 8 * h, row = u * kPage + t;
                    const uint32_t f = __shfl_sync(0xffffffffu, packed, t);
                    const uint32_t fh = __byte_perm(f, f, 0x1010), fl = __byte_perm(f, f, 0x3232);
                    const uint32_t x[4] = {kc[h].x, kc[h].y, kc[h].z, kc[h].w};
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t o[4];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint32_t y, z;
                            e4m3x4_to_f16x2x2(x[2 * e + k], y, z);
                            o[2 * k] = hfma2(y, fh, hmul2(y, fl));
                            o[2 * k + 1] = hfma2(z, fh, hmul2(z, fl));
                        }
                        *reinterpret_cast<uint4 *>(sK + row * 128 + (((2 * (lane & 3) + e) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
                {  // V: element d = lane + 32 h, the tile's 16 tokens
                    const int d = lane + 32 * h;
                    const uint32_t x[4] = {vc[h].x, vc[h].y, vc[h].z, vc[h].w};
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t o[4];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint32_t y, z;
                            e4m3x4_to_f16x2x2(x[2 * e + k], y, z);
                            o[2 * k] = hmul2(y, vf[4 * e + 2 * k]);
                            o[2 * k + 1] = hmul2(z, vf[4 * e + 2 * k + 1]);
                        }
                        *reinterpret_cast<uint4 *>(sV + d * 128 + (((2 * u + e) ^ (d & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(kv_full + 8 * st);
            if ((st += 2) >= kT8Stages) {
                st -= kT8Stages;
                st_ph ^= 1u;
            }
            if ((rs += 2) >= kT8Raw) {
                rs -= kT8Raw;
                rs_ph ^= 1u;
            }
        }
    } else if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 13) asm volatile("griddepcontrol.wait;" ::: "memory");  // (also without units: the kernels after wait for this one alone)
        if (warp == 13 && units > 0) {
            // ---- copies: lane u < 4 the block of tile u of every unit
            const uint64_t policy = evict_first_policy();
            T8Walk w;
            w.start(p, s_start, s_range);
            int wu = w.u0;
            // the block-table entry of the next copy is read one copy early; -2: past the segment's tiles
            auto page_of = [&]() {
                const int k = wu * kT8Tiles + lane;
                // (a bad entry must not pass for "past": -1 stands for all negative ones)
                return lane < kT8Tiles && k < w.keys.ntiles
                           ? max(-1, __ldg(p.block_table + static_cast<size_t>(w.b) * p.max_pages + w.keys.pt_lo + k)) : -2;
            };
            int page = page_of(), rs = 0;
            uint32_t rs_ph = 1;  // (the first round is free)
            const int all = units_of(2);
            failed = all < units;
            int i = 0;
            for (; i < all; ++i) {
                if (__any_sync(0xffffffffu, !mbar_wait_idle(raw_empty + 8 * rs, rs_ph))) {
                    failed = true;
                    break;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the teams have read what was there
                const bool there = page >= 0 && page < p.num_pages;
                if (page != -2 && !there) flag_status(DA_STATUS_BAD_PAGE);  // its tokens read as zeros
                if (lane < kT8Tiles) {
                    const int pos0 = (w.keys.pt_lo + wu * kT8Tiles + lane) * kPage;
                    s_keys[rs][lane] = (there ? max(0, w.keys.lo - pos0) | min(kPage, w.keys.end - pos0) << 8 : 0) | (wu == w.u0 ? 1 << 16 : 0);
                }
                const int copies = __popc(__ballot_sync(0xffffffffu, there));
                __syncwarp();
                const uint32_t bar = raw_full + 8 * rs;
                if (lane == 0) mbar_expect_tx(bar, copies * kBlk8Bytes);
                __syncwarp();
                if (there) {
                    const uint8_t *src = kv + (static_cast<size_t>(page) * p.Hkv + w.g) * kBlk8Bytes;
                    const uint32_t dst = smem_addr(sRaw + (rs * kT8Tiles + lane) * kBlk8Bytes);
                    if (p.row_blocks == 1)  // (64 x 16 tokens: 164 us, 166 without the hint)
                        bulk_load_hint(dst, src, kBlk8Bytes, bar, policy);
                    else  // other row blocks read it too
                        bulk_load(dst, src, kBlk8Bytes, bar);
                }
                if (++wu >= w.u1 && i + 1 < units) {
                    w.next(p);
                    wu = w.u0;
                }
                page = page_of();
                if (++rs == kT8Raw) {
                    rs = 0;
                    rs_ph ^= 1u;
                }
            }
            // nothing may still be landing when the CTA leaves: the last copy of every raw block
            for (int k = max(0, i - kT8Raw); k < i; ++k) mbar_wait_idle(raw_full + 8 * (k % kT8Raw), (k / kT8Raw) & 1);
            __syncwarp();
        } else if (warp >= 14 && units > 0) {
            // ---- query rows as fp16 (zeros past the valid ones), 64 by each of the two warps, a segment ahead of the rows
            T8Walk w;
            w.start(p, s_start, s_range);
            bool more = true;
            for (int k = 0; more; ++k) {
                const int buf = k & 1;
                if ((k >= 2 && __any_sync(0xffffffffu, !mbar_wait_idle(q_free + 8 * buf, ((k >> 1) - 1) & 1))) ||
                    (gives_up(4, k) && warp == 14)) {
                    failed = true;
                    break;
                }
                T8Walk ahead = w;
                more = ahead.next(p);
                if (warp == 14 && lane == 0)  // (the rows are past segment k - 3: they have looked at segment k - 2)
                    s_seg[k & 3] = T8Seg{w.b, w.g, w.rb, w.seq.n, w.seq.L - w.seq.n, w.keys.pt_lo, w.u0, w.u1, w.keys.units, more ? 0 : 1, w.begin};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int rl = (warp - 14) * 64 + 32 * h + lane, r = w.rb * kT8Rows + rl, t = r / p.G;
                    const bool ok = t < w.seq.n;
                    const uint4 *src = reinterpret_cast<const uint4 *>(
                        p.q + (ok ? ((static_cast<size_t>(w.b) * p.T + t) * p.Hq + w.g * p.G + (r - t * p.G)) * kD : 0));
                    uint8_t *dst = sQ + buf * kT8QBytes + rl * 128;
#pragma unroll
                    for (int c0 = 0; c0 < 8; c0 += 4) {
                        uint4 v[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) v[c] = ok ? __ldg(src + c0 + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            *reinterpret_cast<uint4 *>(dst + (((c0 + c) ^ (rl & 7)) << 4)) =
                                make_uint4(bf16x2_to_f16x2(v[c].x), bf16x2_to_f16x2(v[c].y), bf16x2_to_f16x2(v[c].z), bf16x2_to_f16x2(v[c].w));
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // read by the tensor cores
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full + 8 * buf);
                w = ahead;
            }
        } else if (warp == 12 && units > 0) {
        // ---- MMA issuer: S_i = Q K'_i^T, then O += P_{i-1} V'_{i-1}
        const bool leader = elect_one();
        const uint32_t id_qk = umma_idesc_f16(kT8Rows, kT8Keys), id_pv = umma_idesc_f16(kT8Rows, kD);
        const uint64_t dq = umma_sdesc(smem_addr(sQ), 16, 1024), dk = umma_sdesc(smem_addr(sKV), 16, 1024);
        const uint64_t dv = umma_sdesc(smem_addr(sKV) + kT8HalfBytes, 16, 1024);
        auto wait_all = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait_idle(bar, parity)); };
        int seg = -1;
        bool fresh = false, fresh_before = false;  // unit i, i - 1 is its segment's first
        for (int i = 0; i <= units && !failed; ++i) {
            if (i < units) {
                // (S_i's buffer was read before P_{i-2} arrived, which PV_{i-2} below waited for)
                const int s = i % kT8Stages, sb = i & 1;
                if (!wait_all(kv_full + 8 * s, (i / kT8Stages) & 1)) {
                    failed = true;
                    break;
                }
                fresh = __float_as_int(s_fac[s * kT8Tiles].w) != 0;
                if (fresh) {
                    if (leader && seg >= 0) umma_commit(q_free + 8 * (seg & 1));  // the last segment's products are all issued
                    __syncwarp();
                    ++seg;
                    if (!wait_all(q_full + 8 * (seg & 1), (seg >> 1) & 1) || gives_up(3, seg)) {
                        failed = true;
                        break;
                    }
                }
                tc_fence_after();
                if (leader) {
                    const uint64_t dqs = dq + (seg & 1) * (kT8QBytes / 16), dks = dk + s * (kT8StageBytes / 16);
#pragma unroll
                    for (int kk = 0; kk < kD / 16; ++kk)
                        umma_bf16_ss(tm + kT8ColS + 64 * sb, dqs + 2 * kk, dks + 2 * kk, id_qk, kk > 0);
                    umma_commit(s_full + 8 * sb);
                    mbar_arrive(s_full + 8 * sb);  // the rows see what kv_full told this thread: the pages' factors
                }
                __syncwarp();
            }
            if (i >= 1) {
                const int j = i - 1, s = j % kT8Stages, pb = j & 1;
                if (!wait_all(p_full + 8 * pb, (j >> 1) & 1)) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                if (leader) {
                    const uint64_t dvs = dv + s * (kT8StageBytes / 16);
#pragma unroll
                    for (int kk = 0; kk < kT8Keys / 16; ++kk)
                        umma_bf16_ts(tm + kT8ColO, tm + kT8ColP + 32 * pb + 8 * kk, dvs + 2 * kk, id_pv, kk > 0 || !fresh_before ? 1u : 0u);
                    umma_commit(o_done + 8 * pb);
                    umma_commit(kv_empty + 8 * s);
                }
                __syncwarp();
            }
            fresh_before = fresh;
        }
        if (leader) {
            umma_commit(drain);  // completes when every MMA issued above has
            mbar_wait_bounded(drain, 0);
        }
        __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 88;");
        // ---- query rows: one per thread
        if (units > 0) {
        const uint32_t lanes = static_cast<uint32_t>(32 * warp) << 16;
        int i = 0, st = 0;
        float R = -INFINITY;
        for (int seg = 0; !failed; ++seg) {
            int pr, lor, jf, count;  // the row's keys [lor, pr], the unit's first position, the segment's units here
            bool valid, warp_active;
            int place;  // the row's among its sequence's output rows, or -1
            float sink = -INFINITY;
            if (warp == 0 && gives_up(0, seg)) {
                failed = true;
                break;
            }
            if (__any_sync(0xffffffffu, !mbar_wait_bounded(q_full + 8 * (seg & 1), (seg >> 1) & 1))) {
                failed = true;
                break;
            }
            {
                const T8Seg &w = s_seg[seg & 3];
                const int r = w.rb * kT8Rows + tid, r_valid = w.n * p.G, t = r / p.G;
                place = t < p.T ? t * p.Hq + w.g * p.G + (r - t * p.G) : -1;
                valid = r < r_valid;
                warp_active = w.rb * kT8Rows + 32 * warp < r_valid;
                pr = valid ? w.base + t : -1;
                lor = valid && p.window > 0 ? max(0, w.base + t - p.window + 1) : 0;
                jf = (w.pt_lo + w.u0 * kT8Tiles) * kPage;
                count = w.u1 - w.u0;
                if (valid && p.sinks != nullptr) sink = __ldg(p.sinks + w.g * p.G + (r - t * p.G));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(q_free + 8 * (seg & 1));
            float l = 0.f;
            for (int k = 0; k < count && !failed; ++k, ++i, jf += kT8Keys) {
                const int sb = i & 1;
                // every row warp waits for S_i, rows or not, so that no warp's arrival on p_full can run ahead
                // into a later phase (a give-up is taken by the whole warp: the TMEM accesses are warp-wide)
                if (__any_sync(0xffffffffu, !mbar_wait_bounded(s_full + 8 * sb, (i >> 1) & 1))) {
                    failed = true;
                    break;
                }
                if (warp_active) {
                    // (S_i complete: so is PV_{i-2}, which read the P buffer)
                    tc_fence_after();
                    const uint32_t sc = tm + lanes + kT8ColS + 64 * sb, pc = tm + lanes + kT8ColP + 32 * sb;
                    const float4 *fac = s_fac + st * kT8Tiles;
                    const bool interior = __all_sync(0xffffffffu, jf >= lor && jf + kT8Keys - 1 <= pr);
                    const int a = lor - jf, e = pr + 1 - jf;  // keys [a, e) of the unit are this row's
                    // one tile's scores; keys that are not the row's: -inf
                    auto mask = [&](int u, uint32_t(&x)[16]) {
                        if (!interior) {
#pragma unroll
                            for (int c = 0; c < 16; ++c)
                                if (16 * u + c < a || 16 * u + c >= e) x[c] = 0xff800000u;
                        }
                    };
                    float l_unit;
                    // a tile's probabilities with the reference R into P, and their sum
                    auto tile = [&](int u, uint32_t(&x)[16]) {
                        mask(u, x);
                        const float2 f = *reinterpret_cast<const float2 *>(fac + u);
                        const float ad = f.y + (kT8Shift - (R == -INFINITY ? 0.f : R));
                        const float2 mul = make_float2(f.x, f.x), add = make_float2(ad, ad);
                        float2 ls[2] = {{0.f, 0.f}, {0.f, 0.f}};
                        uint32_t pk[8];
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const float2 y = fma2(make_float2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), mul, add);
                            const float a0 = fast_exp2(y.x), a1 = fast_exp2(y.y);
                            ls[c & 1] = add2(ls[c & 1], make_float2(a0, a1));
                            pk[c] = pack_f16(a0, a1);
                        }
                        tmem_st8(pc + 8 * u, pk);
                        return add2(ls[0], ls[1]);
                    };
                    // (a tile's scores are fetched while the one before is worked on; the sums are looked at at the end, where
                    // their latencies overlap); the largest tile's sum
                    auto probabilities = [&]() {
                        uint32_t x0[16], x1[16];
                        tmem_ld16(sc, x0);
                        tmem_wait_ld();
                        tmem_ld16(sc + 16, x1);
                        const float2 s0 = tile(0, x0);
                        tmem_wait_ld();
                        tmem_ld16(sc + 32, x0);
                        const float2 s1 = tile(1, x1);
                        tmem_wait_ld();
                        tmem_ld16(sc + 48, x1);
                        const float2 s2 = tile(2, x0);
                        tmem_wait_ld();
                        const float2 s3 = tile(3, x1);
                        const float t0 = s0.x + s0.y, t1 = s1.x + s1.y, t2 = s2.x + s2.y, t3 = s3.x + s3.y;
                        l_unit = fmaf(t0, fac[0].z, t1 * fac[1].z) + fmaf(t2, fac[2].z, t3 * fac[3].z);
                        return fmaxf(fmaxf(t0, t1), fmaxf(t2, t3));
                    };
                    bool need = R == -INFINITY && valid;
                    if (!__any_sync(0xffffffffu, need)) {
                        // a segment's first unit is tried with the last one's reference (mostly the same head's, a few tokens
                        // before), kept where the probabilities have not sunk in fp16's range
                        const float top = probabilities();
                        need = top > kT8TileMax || (k == 0 && valid && !(top >= 16.f));
                    }
                    if (__any_sync(0xffffffffu, need)) {
                        float mb = -INFINITY;
#pragma unroll 1
                        for (int u = 0; u < kT8Tiles; ++u) {
                            uint32_t x[16];
                            tmem_ld16(sc + 16 * u, x);
                            tmem_wait_ld();
                            mask(u, x);
                            const float4 f = fac[u];
                            float mt = -INFINITY;
#pragma unroll
                            for (int c = 0; c < 16; c += 2) mt = max3(mt, __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
                            mb = fmaxf(mb, fmaf(mt, f.x, f.y));  // the multiplier is positive
                        }
                        // (also where a row without a reference called for this, and nothing was tried)
                        need = need || (valid && (k == 0 || mb > R + kT8Ahead));
                        const float Rn = need ? (k == 0 ? ceilf(mb) : fmaxf(R, ceilf(mb))) : R;  // an integer: F - R and the rescaling are exact
                        const float f = k == 0 || Rn == R ? 1.f : exp2f(R - Rn);  // R = -inf: 0 (O and l are 0)
                        if (k > 0) {
                            // O holds the segment's PVs up to PV_{i-1}, whose barrier cannot be a phase further:
                            // PV_{i+1} waits for P_{i+1}
                            if (__any_sync(0xffffffffu, !mbar_wait_bounded(o_done + 8 * (sb ^ 1), ((i - 1) >> 1) & 1))) {
                                failed = true;
                                break;
                            }
                            tc_fence_after();
#pragma unroll 1
                            for (int h = 0; h < 4; ++h) {
                                uint32_t o[16];
                                tmem_ld16(tm + lanes + kT8ColO + 16 * h, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
                                tmem_st16(tm + lanes + kT8ColO + 16 * h, o);
                                tmem_wait_st();
                            }
                        }
                        l *= f;
                        R = Rn;
                        tmem_wait_st();
                        probabilities();
                    }
                    l += l_unit;
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * sb);
                if (++st == kT8Stages) st = 0;
            }
            // ---- finish this thread's row: O (after the segment's last PV) -> output or partial
            const int last = i - 1;
            if (!failed && warp_active && __any_sync(0xffffffffu, !mbar_wait_bounded(o_done + 8 * (last & 1), (last >> 1) & 1)))
                failed = true;
            if (failed) break;
            const T8Seg &w = s_seg[seg & 3];
            if (l == 0.f) R = -INFINITY;  // no key of the row here
            sink *= kLog2e;
            const bool whole = w.u0 == 0 && w.u1 == w.units;
            const float m_row = R - kT8Shift;
            float f = 0.f;  // rows that are not queries: zeros
            if (whole && valid) {
                const float M = fmaxf(m_row, sink);
                if (M != -INFINITY) {
                    const float den = l * exp2f(m_row - M) + (sink == -INFINITY ? 0.f : exp2f(sink - M));
                    f = den > 0.f ? exp2f(m_row - M) / den : den == den ? 0.f : den;
                }
            }
            float *const slot = p.part + (static_cast<size_t>(cta) * 2 + (seg == 0 ? 0 : 1)) * kT8SlotFloats;
            if (!whole && valid) {
                slot[tid] = m_row;
                slot[kT8Rows + tid] = l;
            }
            tc_fence_after();
            uint4 *const dst = reinterpret_cast<uint4 *>(p.out + (static_cast<size_t>(w.b) * p.T * p.Hq + max(place, 0)) * kD);
            auto columns = [&](int h, uint32_t(&x)[16]) {  // columns 16 h .. + 15
                float o[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) o[c] = valid ? __uint_as_float(x[c]) : 0.f;
                if (whole) {
                    if (place >= 0) {
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            dst[2 * h + c] = make_uint4(pack_bf16(o[8 * c] * f, o[8 * c + 1] * f), pack_bf16(o[8 * c + 2] * f, o[8 * c + 3] * f),
                                                        pack_bf16(o[8 * c + 4] * f, o[8 * c + 5] * f), pack_bf16(o[8 * c + 6] * f, o[8 * c + 7] * f));
                    }
                } else if (valid) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        *const_cast<float4 *>(t8_acc(slot, 4 * h + c, tid)) = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
                }
            };
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                uint32_t x[16] = {};
                if (warp_active) {
                    tmem_ld16(tm + lanes + kT8ColO + 16 * h, x);
                    tmem_wait_ld();
                }
                columns(h, x);
            }
            tc_fence_before();  // (the next segment's first PV writes O after this warp's next P)
            if (!whole && !p.defer && __any_sync(0xffffffffu, place >= 0)) {
                // the last of the CTAs that share the segment folds its partials, every warp its own 32 rows: a
                // counter per warp, at the segment's first CTA (which has no other segment that goes on)
                const long long U = s_range[2];
                const int c0 = t8_owner(U, nc, w.begin), c1 = t8_owner(U, nc, w.begin + w.units - 1);
                __threadfence();
                __syncwarp();
                int ticket = 0;
                if (lane == 0) ticket = atomicAdd(p.counters + 4 * c0 + warp, 1);
                if (__shfl_sync(0xffffffffu, ticket, 0) == c1 - c0) {
                    __threadfence();
                    if (place >= 0)
                        t8_fold(p, c0, t8_first(U, nc, c0) < w.begin - kT8SegCost ? 1 : 0, c1 - c0 + 1, tid, place % p.Hq, valid, dst);
                }
            }
            if (w.last) break;
        }
        }
    }
    if (failed) flag_status(DA_STATUS_TIMEOUT);

    // ---- teardown: every MMA done (the issuer has waited) before TMEM is released
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(kT8TmemCols));
    }
}

// The partials of the segments that several CTAs share, folded after the attention: where few segments are spread over
// the whole grid the CTA that comes last would fold dozens alone. One CTA per 32 rows of a segment; a thread has a row,
// and each of the eight warps every eighth partial; the warps' sums meet in shared memory. The split is worked
// out again from the lengths.
constexpr int kT8FoldWarps = 8;
__global__ void __launch_bounds__(kT8FoldWarps * 32) t8_combine_kernel(const MultiParams p, int grid) {
    __shared__ union {
        long long pre[kMaxBatch + 1];
        float sum[kT8FoldWarps][32][17];
    } sh;
    __shared__ float s_m[kT8FoldWarps][32], s_l[kT8FoldWarps][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rb = blockIdx.x / 4, rl = blockIdx.x % 4 * 32 + lane;
    const int g = blockIdx.y, b = blockIdx.z;
    const T8Seq s = t8_seq(p, b);
    if (rb >= s.blocks) return;  // zeros, written by the attention
    t8_prefix(p, sh.pre, nullptr, warp, kT8FoldWarps, lane);
    const long long U = sh.pre[p.B];
    const int nc = t8_ctas(U, grid);
    long long begin = sh.pre[b] + (sh.pre[b + 1] - sh.pre[b]) / p.Hkv * g;
    for (int i = 0; i < rb; ++i) begin += t8_cost(p, s, i);
    begin += kT8SegCost;
    const int c0 = t8_owner(U, nc, begin), c1 = t8_owner(U, nc, begin + t8_keys(p, s, rb).units - 1);
    const int r0 = rb * kT8Rows;
    if (c0 == c1 || r0 + blockIdx.x % 4 * 32 >= p.T * p.G) return;
    const int count = c1 - c0 + 1, k0 = t8_first(U, nc, c0) < begin - kT8SegCost ? 1 : 0;
    const int r = r0 + rl, t = r / p.G, hl = r - t * p.G;
    const bool row = r < p.T * p.G, query = row && t < s.n;
    float M = -INFINITY;
    if (query) {
#pragma unroll 4
        for (int i = warp; i < count; i += kT8FoldWarps) M = fmaxf(M, __ldcg(t8_slot(p, c0, k0, i) + rl));
    }
    s_m[warp][lane] = M;
    __syncthreads();  // (and the prefix has been read)
    const float sg = query && p.sinks != nullptr ? __ldg(p.sinks + g * p.G + hl) * kLog2e : -INFINITY;
    float Mf = sg;
#pragma unroll
    for (int w = 0; w < kT8FoldWarps; ++w) Mf = fmaxf(Mf, s_m[w][lane]);
    float d = 0.f;
    float4 o[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (query && Mf != -INFINITY)
        for (int i = warp; i < count; i += kT8FoldWarps) {
            const float *sl = t8_slot(p, c0, k0, i);
            const float m = __ldcg(sl + rl);
            if (m == -INFINITY) continue;  // no key of the row there
            const float w = exp2f(m - Mf);
            d += __ldcg(sl + kT8Rows + rl) * w;
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const float4 x = __ldcg(t8_acc(sl, c, rl));
                o[c].x += x.x * w, o[c].y += x.y * w, o[c].z += x.z * w, o[c].w += x.w * w;
            }
        }
    s_l[warp][lane] = d;
    float den = 0.f, inv = 0.f;
    uint32_t *out = reinterpret_cast<uint32_t *>(p.out + ((static_cast<size_t>(b) * p.T + t) * p.Hq + g * p.G + hl) * kD);
#pragma unroll
    for (int h = 0; h < 4; ++h) {  // 16 columns at a time; this thread adds up columns 2 warp, 2 warp + 1 of its row
        __syncthreads();
        if (h == 0) {
            den = sg == -INFINITY ? 0.f : exp2f(sg - Mf);
#pragma unroll
            for (int w = 0; w < kT8FoldWarps; ++w) den += s_l[w][lane];
            inv = den > 0.f ? 1.f / den : den == den ? 0.f : den;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float *x = &sh.sum[warp][lane][4 * c];
            x[0] = o[4 * h + c].x, x[1] = o[4 * h + c].y, x[2] = o[4 * h + c].z, x[3] = o[4 * h + c].w;
        }
        __syncthreads();
        float x0 = 0.f, x1 = 0.f;
#pragma unroll
        for (int w = 0; w < kT8FoldWarps; ++w) {
            x0 += sh.sum[w][lane][2 * warp];
            x1 += sh.sum[w][lane][2 * warp + 1];
        }
        if (row) out[8 * h + warp] = pack_bf16(x0 * inv, x1 * inv);
    }
}
