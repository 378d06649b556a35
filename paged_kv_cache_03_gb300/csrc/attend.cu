// attend.cu -- the cache attention's host side: which kernel takes a call, the
// workspace, the launches.
#include <algorithm>

#include "walk.cuh"

namespace pa {

using namespace walk;

namespace {

struct WalkPlan {
    int R, nt, nrc, rows_cta;  // nt: n-tiles of 8 rows of walk_kernel, 0: block_kernel
    bool whole;                // walk_kernel: a CTA per segment
    bool scores;               // key weights from stored scores
    long long items;           // CTAs
    size_t split_off, ml_off, o_off, lse_off, score_off, total;  // score_off: scores, or the packed query
};

// Rows per kv head from which block_kernel takes a call (walk, block, us, fp32 queries:
// B = 8 over 1000 .. 8000 keys 61, 69 at 32 rows, 84, 71 at 48; B = 64 over 500 .. 2000
// keys 130, 143 at 32, 186, 147 at 48; B = 1 over 16000 keys 49, 49 at 64; both since 2 us
// more, for the low parts' own range).
constexpr int kBlockRows = 48;
// Key weights: rows per kv head up to which scores are stored, and the most bytes of them
// (4 for every slot of the table and row: a wide table would take more than the cache);
// otherwise the weights are recomputed from the keys (stored, recomputed, us, 64 sequences
// of 128 .. 4096 keys, 4 rows, 8 kv heads: 4-bit pages 60, 122, and 93, 194 in tables of
// 32768 slots, 268 MB of scores; bf16 pages 120, 169, and 153, 243).
constexpr int kScoreRows = 8;
constexpr size_t kScoreBytes = size_t(1) << 29;
// Table capacity up to which a CTA takes a whole segment, without a merge (shares,
// whole, us, G = 4, H_kv = 8): 64 sequences of 1000 keys 30, 23, one of 1000 18, 16,
// one of 2000 18, 18, one of 4000 18, 34.
constexpr int kWholeKeys = 1024;
constexpr int kMinPer = 2;       // least cost of a share

// walk_kernel: 8 rows per CTA, or 16 where a (sequence, kv head) has more than
// 8 (not for fp32 queries, whose fragments take twice the registers); block_kernel:
// 64.  As many CTAs as are resident together, each an equal share of all keys, or,
// over short tables, one per segment and no merge.
WalkPlan plan(const pa_shape& sh, bool q4, bool weights, int sm_count) {
    WalkPlan w;
    w.R = sh.H_q / sh.H_kv * sh.L;
    const bool f32 = sh.dtype == PA_F32;
    w.nt = w.R >= kBlockRows ? 0 : w.R > 8 && !f32 ? 2 : 1;
    w.rows_cta = w.nt ? 8 * w.nt : kBlockCtaRows;
    w.nrc = (w.R + w.rows_cta - 1) / w.rows_cta;
    const long long cap = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    const long long segs = static_cast<long long>(sh.B) * sh.H_kv * w.nrc;
    const size_t rows = static_cast<size_t>(sh.B) * sh.H_kv * w.R;
    w.scores = weights && w.R <= kScoreRows && rows * cap * 4 <= kScoreBytes;
    w.whole = w.nt && cap <= kWholeKeys;
    const int resident = w.nt ? walk_resident(w.nt, q4, f32, w.R) : 2;
    w.items = w.whole ? segs : static_cast<long long>(sm_count) * resident;
    const size_t slots = w.whole ? 0 : static_cast<size_t>(w.items) * 2 * w.rows_cta;
    size_t off = kFlagBytes;
    w.split_off = off;
    if (!w.whole) off = align_up(off + static_cast<size_t>(w.items) * 16, 256);
    w.ml_off = off;
    off = align_up(off + slots * 16, 256);
    w.o_off = off;
    off = align_up(off + slots * kD * 4, 256);
    w.lse_off = off;
    if (weights) off = align_up(off + rows * 4, 256);
    w.score_off = off;
    if (weights) off = align_up(off + (w.scores ? rows * cap * 4 : weights_scratch_bytes(sh, sm_count)), 256);
    w.total = off;
    return w;
}

// The attention, its merge over shares, then the key weights.
pa_status launch(const WalkParams& p, const WalkPlan& w, bool q4, bool f32, const DeviceInfo& dev, void* scratch,
                 cudaStream_t stream) {
    const long long bk = static_cast<long long>(p.B) * p.H_kv;
    if (w.items > INT_MAX || bk * p.R > INT_MAX) return PA_ERR_UNSUPPORTED;
    // the shares count costs in an int
    if (!w.whole && bk * p.nrc * (p.max_S / kUnit + 1 + kSegCost) > INT_MAX / 2) return PA_ERR_UNSUPPORTED;
    const WalkLaunch l = {w.nt, q4, f32, w.items, dev.device, stream};
    pa_status st = w.nt ? walk_attend(p, l) : block_attend(p, l);
    if (st == PA_OK && !w.whole) st = merge_shares(p, w.rows_cta, static_cast<int>(w.items), f32, stream);
    if (st != PA_OK || !p.w_out) return st;
    return w.scores ? weights_from_scores(p, stream) : weights_from_keys(p, q4, f32, scratch, dev, stream);
}

// Rows per kv head from which bf16 queries go to the tensor-core tiles of tiles.cu: fewer
// where the keys of all (sequence, kv head) are many.  Measured (walk or block, tiles, us;
// G = 4, H_kv = 8).  4-bit pages, 40 rows: 64 sequences of 500 .. 2000 keys 115, 98; 8 of
// 1000 .. 8000 55, 49; one of 16000 33, 33; 2 of 900 16, 25; 32 rows: 86, 98; 43, 49; 27, 33.
// At 56 rows 2 of 900 22, 25.  bf16 pages with key weights, 20 rows: 171, 138; 79, 79; one of
// 16000 42, 46, at 40 50, 48; 2 of 500 18, 30.
constexpr int kTileRows = 64, kTileRowsMany = 40, kTileRowsManyBf16 = 20;
constexpr long long kManyKeys = 1 << 17, kManyKeysBf16 = 1 << 18;

bool tiles_take(const pa_shape& sh, bool q4, int sm_count) {
    const long long R = static_cast<long long>(sh.H_q / sh.H_kv) * sh.L;
    const long long keys = static_cast<long long>(sh.B) * sh.H_kv * sh.max_pages_per_seq * sh.page_size;
    const bool many = keys >= (q4 ? kManyKeys : kManyKeysBf16);
    return sh.dtype == PA_BF16 && R >= (!many ? kTileRows : q4 ? kTileRowsMany : kTileRowsManyBf16) &&
           tiles_supported(sh, sm_count);
}

// ---- whole prompts over 4-bit pages: bf16 copies and the bf16 tile kernel -------
// (K and V exact: a 4-bit value is a bf16 number; P rounded to bf16 as over bf16 pages,
// where the other kernels round it to f16: whole prompts 0.0020 from 64 bits, relative,
// against 0.0017, of which 0.0016 is the bf16 output).  Where a kv head has half as many rows as
// keys or more, the copies cost less than what tiles.cu spends per segment
// (G = 4, H_kv = 8, us, tiles against copies: 4 x 2048 rows over 600 keys 46, 38; 4 x
// 8192 over 2048 198, 145; 8 x 2080 over 1000 .. 8000 352, 382; 8 x 1040 209, 247; 1 x
// 8192 over 16000 436, 444).  Sequences go in groups whose copies fit kDenseBytes.
constexpr size_t kDenseBytes = size_t(1) << 30;

struct DensePlan {
    pa_shape sh;  // one group, over the dense copies
    size_t id_off, k_off, v_off, total;  // id: block table, then lengths
};

bool dense_take(const pa_shape& sh, bool q4, bool weights, int sm_count, DensePlan* t) {
    if (!q4 || weights || sh.dtype != PA_BF16) return false;
    const long long cap = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    const long long R = static_cast<long long>(sh.H_q / sh.H_kv) * sh.L;
    if (R < kTileRows || 2 * R < cap) return false;
    const long long slots = (cap + 127) / 128 * 128;
    const size_t per_seq = static_cast<size_t>(slots) * sh.H_kv * kD * 2 * 2;
    if (slots * sh.H_kv >= (1ll << 31)) return false;
    long long nb = static_cast<long long>(kDenseBytes / per_seq);
    nb = nb < 1 ? 1 : nb < sh.B ? nb : sh.B;
    t->sh = sh;
    t->sh.B = static_cast<int>(nb);
    t->sh.num_pages = t->sh.B;
    t->sh.page_size = static_cast<int>(slots);
    t->sh.max_pages_per_seq = 1;
    if (!prefill_supported(t->sh)) return false;
    size_t off = tile_partials_offset(t->sh, sm_count) + tile_partial_bytes(t->sh, sm_count);
    pa_shape last = t->sh;  // the last group may split its keys more
    last.B = sh.B % last.B > 0 ? sh.B % last.B : last.B;
    const size_t off_last = tile_partials_offset(last, sm_count) + tile_partial_bytes(last, sm_count);
    t->id_off = off = align_up(off > off_last ? off : off_last, 256);
    off = align_up(off + 8 * static_cast<size_t>(nb), 256);
    t->k_off = off;
    off += nb * per_seq / 2;
    t->v_off = off;
    t->total = off + nb * per_seq / 2;
    return true;
}

pa_status dense_launch(const WalkCall& c, const DensePlan& t) {
    const pa_shape& sh = c.sh;
    uint8_t* const ws = static_cast<uint8_t*>(c.ws);
    const pa_q4_pool pool = {const_cast<void*>(c.kc), const_cast<void*>(c.ks), const_cast<void*>(c.vc),
                             const_cast<void*>(c.vs)};
    const size_t per_seq = static_cast<size_t>(sh.H_q) * sh.L * kD * 2;  // query and output bytes
    for (int b0 = 0; b0 < sh.B; b0 += t.sh.B) {
        const int nb = t.sh.B < sh.B - b0 ? t.sh.B : sh.B - b0;
        pa_shape src = sh;
        src.B = nb;
        pa_status st = q4_gather_launch(src, pool, c.bt + static_cast<long long>(b0) * sh.max_pages_per_seq,
                                        c.ctx + b0, t.sh.page_size, 0, 0,
                                        reinterpret_cast<int32_t*>(ws + t.id_off), t.sh.B, ws + t.k_off, ws + t.v_off,
                                        reinterpret_cast<uint32_t*>(ws), c.stream);
        if (st != PA_OK) return st;
        Call d;
        d.sh = t.sh;
        d.sh.B = nb;
        d.q = static_cast<const uint8_t*>(c.q) + b0 * per_seq;
        d.kp = ws + t.k_off;
        d.vp = ws + t.v_off;
        d.bt = reinterpret_cast<const int32_t*>(ws + t.id_off);
        d.ctx = d.bt + t.sh.B;
        d.scale = c.scale;
        d.causal = c.causal;
        d.out = static_cast<uint8_t*>(c.out) + b0 * per_seq;
        d.ws = c.ws;
        d.ws_bytes = t.id_off;
        d.stream = c.stream;
        d.dev = c.dev;
        st = prefill_launch(d);
        if (st != PA_OK) return st;
    }
    return PA_OK;
}

}  // namespace

// Where the weights' scratch lies: after the tiles' own part and the log-sum-exps.
static size_t tiles_scratch(const pa_shape& sh, int sm_count) {
    return align_up(align_up(tiles_workspace_bytes(sh, sm_count), 256) + static_cast<size_t>(sh.B) * sh.H_q * sh.L * 4, 256);
}

// What this very shape needs.
static size_t needed_bytes(const pa_shape& sh, bool q4, bool weights, int sm_count) {
    DensePlan d;
    if (dense_take(sh, q4, weights, sm_count, &d)) return d.total;
    if (tiles_take(sh, q4, sm_count)) {
        const size_t n = align_up(tiles_workspace_bytes(sh, sm_count), 256);
        return weights ? tiles_scratch(sh, sm_count) + weights_scratch_bytes(sh, sm_count) : n;
    }
    return plan(sh, q4, weights, sm_count).total;
}

// The most that a call of at most this B, L and max_pages_per_seq needs.  Which kernel takes
// a call is not monotone in them (a decode step stores scores, a chunk does not), so each
// part is counted for every kernel that some smaller call may take, at its largest.
size_t walk_workspace_bytes(const pa_shape& sh, bool q4, bool weights, int sm_count) {
    const size_t cap = static_cast<size_t>(sh.max_pages_per_seq) * sh.page_size, sms = static_cast<size_t>(sm_count);
    const size_t G = sh.H_q / sh.H_kv, R = G * sh.L, bk = static_cast<size_t>(sh.B) * sh.H_kv, rows = bk * R;
    const bool f32 = sh.dtype == PA_F32;
    constexpr size_t kState = 16 + kD * 4;  // of a row: max and sums, O
    const size_t lse = weights ? rows * 4 : 0, scratch = weights ? weights_scratch_most(sh, sm_count) : 0;
    // walk_kernel with 8 or 16 rows a CTA, block_kernel with 64
    auto shares = [&](size_t ctas, size_t rows_cta) { return ctas * (16 + 2 * rows_cta * kState); };
    size_t few = 0;
    if (cap > kWholeKeys) few = shares(sms * walk_resident(1, q4, f32, 1), 8);
    if (cap > kWholeKeys && R > 8 && !f32) few = std::max(few, shares(sms * walk_resident(2, q4, f32, 16), 16));
    if (R >= kBlockRows) few = std::max(few, shares(sms * 2, kBlockCtaRows));
    size_t scores = 0;
    if (weights && G <= kScoreRows)
        scores = std::min(bk * G * std::min<size_t>(sh.L, kScoreRows / G) * cap * 4, kScoreBytes);
    size_t most = few + lse + std::max(scores, scratch);
    if (!f32 && R >= (q4 ? kTileRowsMany : kTileRowsManyBf16))
        most = std::max(most, tiles_workspace_most(sh, sm_count) + lse + scratch);
    if (q4 && !weights && !f32 && R >= kTileRows) {  // bf16 copies of up to 2 R keys
        const size_t per_seq = (std::min(cap, 2 * R) + 127) / 128 * 128 * sh.H_kv * kD * 2 * 2;
        const size_t copies = std::max(per_seq, std::min(per_seq * sh.B, kDenseBytes));
        const size_t states = std::max(rows, 256 * sms + 128 * bk) + 256 * bk;  // key chunks, a short last tile
        most = std::max(most, tile_partials_offset(sh, sm_count) + states * kState + 8 * static_cast<size_t>(sh.B) + copies);
    }
    most = align_up(kFlagBytes + most + 16 * 256, 256);  // (each part starts on 256 bytes)
    return std::max(most, needed_bytes(sh, q4, weights, sm_count));
}

pa_status walk_launch(const WalkCall& c) {
    const pa_shape& sh = c.sh;
    const bool tiles = tiles_take(sh, c.ks != nullptr, c.dev.sm_count);
    const WalkPlan w = plan(sh, c.ks != nullptr, c.w_out != nullptr, c.dev.sm_count);
    if (c.w_out && !weights_supported(sh, c.w_S, c.dev.sm_count)) return PA_ERR_UNSUPPORTED;
    if (c.ws_bytes < needed_bytes(sh, c.ks != nullptr, c.w_out != nullptr, c.dev.sm_count)) return PA_ERR_WORKSPACE;
    uint8_t* const ws = static_cast<uint8_t*>(c.ws);
    WalkParams p;
    p.q = c.q;
    p.kc = c.kc;
    p.vc = c.vc;
    p.ks = c.ks;
    p.vs = c.vs;
    p.bt = c.bt;
    p.ctx = c.ctx;
    p.out = c.out;
    p.part_ml = reinterpret_cast<float4*>(ws + w.ml_off);
    p.part_o = reinterpret_cast<float*>(ws + w.o_off);
    p.lse = c.w_out ? reinterpret_cast<float*>(ws + w.lse_off) : nullptr;
    p.w_in = c.w_in;
    p.w_out = c.w_out;
    p.w_S = c.w_S;
    p.flag = reinterpret_cast<uint32_t*>(ws);
    p.B = sh.B;
    p.H_kv = sh.H_kv;
    p.L = sh.L;
    p.R = w.R;
    p.num_pages = sh.num_pages;
    p.ps = sh.page_size;
    p.max_npg = sh.max_pages_per_seq;
    p.causal = c.causal;
    p.nrc = w.nrc;
    p.whole = w.whole ? 1 : 0;
    p.min_per = kMinPer;
    p.split = reinterpret_cast<int4*>(ws + w.split_off);
    p.max_S = static_cast<long long>(sh.max_pages_per_seq) * sh.page_size;
    p.scale_log2 = c.scale * 1.4426950408889634f;
    p.score = w.scores ? reinterpret_cast<float*>(ws + w.score_off) : nullptr;
    p.cap = p.max_S;
    DensePlan d;
    if (dense_take(sh, c.ks != nullptr, c.w_out != nullptr, c.dev.sm_count, &d)) return dense_launch(c, d);
    if (tiles) {
        void* const scratch = ws + tiles_scratch(sh, c.dev.sm_count);
        if (c.w_out)
            p.lse = reinterpret_cast<float*>(ws + align_up(tiles_workspace_bytes(sh, c.dev.sm_count), 256));
        const pa_status st = tiles_launch(c, p.lse);
        return st != PA_OK || !c.w_out ? st : weights_from_keys(p, c.ks != nullptr, false, scratch, c.dev, c.stream);
    }
    return launch(p, w, c.ks != nullptr, sh.dtype == PA_F32, c.dev, ws + w.score_off, c.stream);
}

}  // namespace pa
