// decode.cpp -- the C entry points of libred_decode.h: argument checks,
// launch shapes, and the calls into the kernels.
#include "decode.hpp"

#include <initializer_list>
#include <optional>

#include "decode_host.hpp"
#include "libred_serve.h"

using namespace libred;

namespace {

bool heads_valid(const red_heads& h, size_t tokens, size_t dim, size_t esize) {
    const int64_t s = span_of(h, tokens, dim);
    if (s < 0) return false;
    return s == 0 || (h.data != nullptr && is_aligned(h.data, esize));
}

bool spans_meet(const red_heads& a, const red_heads& b, size_t tokens, size_t dim, size_t esize) {
    const uintptr_t as = (uintptr_t)span_of(a, tokens, dim) * esize, bs = (uintptr_t)span_of(b, tokens, dim) * esize;
    const uintptr_t a0 = (uintptr_t)a.data, b0 = (uintptr_t)b.data;
    return as && bs && a0 < b0 + bs && b0 < a0 + as;
}

bool same_place(const red_heads& a, const red_heads& b) {
    return a.data == b.data && a.token_stride == b.token_stride && a.head_stride == b.head_stride;
}

// An output over its own input: the same rows, or none of them.
bool output_valid(const red_heads& out, const red_heads& in, size_t tokens, size_t dim, size_t esize) {
    if (out.heads != in.heads || !heads_valid(out, tokens, dim, esize) || !rows_apart(out, tokens, dim)) return false;
    return same_place(out, in) || !spans_meet(out, in, tokens, dim, esize);
}

Heads to_heads(const red_heads& h) { return Heads{h.data, h.token_stride, h.head_stride}; }

// Whether rows can be read `bytes` at a time: rows start on such a boundary.
bool rows_on(const red_heads& h, size_t tokens, size_t esize, size_t bytes) {
    if (h.heads == 0) return true;
    return is_aligned(h.data, bytes) && (tokens <= 1 || h.token_stride * (int64_t)esize % (int64_t)bytes == 0) &&
           (h.heads == 1 || h.head_stride * (int64_t)esize % (int64_t)bytes == 0);
}

static_assert(libred::kQkNormWaves == 4 && libred::kCacheWaves == 4, "blocks of 256 threads");

// Heads from token t on.
Heads heads_from(const red_heads& h, size_t t, size_t esize) {
    return Heads{h.data ? static_cast<char*>(h.data) + (int64_t)t * h.token_stride * (int64_t)esize : nullptr, h.token_stride, h.head_stride};
}

using QkNormLaunch = hipError_t (*)(int, int, const libred::QkNorm&, bool, int, hipStream_t);

red_status qk_norm_call(const red_qk_norm_rope_args* a, const red_heads* dq, const red_heads* dk, float* dqw,
                        float* dkw, bool back, hipStream_t stream) {
    if (a == nullptr || (back && (dq == nullptr || dk == nullptr))) return RED_ERR_INVALID_ARG;
    if (a->type != RED_F32 && a->type != RED_F16 && a->type != RED_BF16) return RED_ERR_INVALID_ARG;
    const size_t es = type_bytes(a->type), T = a->tokens, D = a->dim;
    if (D < 1 || D > RED_HEAD_MAX_DIM || a->rot > D || a->rot % 2 != 0 || T > RED_MAX_N) return RED_ERR_INVALID_ARG;
    if (!(a->eps >= 0.f)) return RED_ERR_INVALID_ARG;
    if (a->q.heads > 1 << 20 || a->k.heads > 1 << 20) return RED_ERR_INVALID_ARG;
    if (!heads_valid(a->q, T, D, es) || !heads_valid(a->k, T, D, es)) return RED_ERR_INVALID_ARG;
    if (!output_valid(a->q_out, a->q, T, D, es) || !output_valid(a->k_out, a->k, T, D, es)) return RED_ERR_INVALID_ARG;
    if (!is_aligned(a->q_weight, es) || !is_aligned(a->k_weight, es)) return RED_ERR_INVALID_ARG;
    if (!is_aligned(a->pos, 8) || !is_aligned(a->freq, 4)) return RED_ERR_INVALID_ARG;
    if (back) {
        if (dq->heads != a->q.heads || dk->heads != a->k.heads) return RED_ERR_INVALID_ARG;
        if (!heads_valid(*dq, T, D, es) || !heads_valid(*dk, T, D, es)) return RED_ERR_INVALID_ARG;
        if (!output_valid(a->q_out, *dq, T, D, es) || !output_valid(a->k_out, *dk, T, D, es)) return RED_ERR_INVALID_ARG;
        if (!is_aligned(dqw, 4) || !is_aligned(dkw, 4)) return RED_ERR_INVALID_ARG;
    }
    const int rows = (int)(a->q.heads + a->k.heads);
    const bool empty = T == 0 || rows == 0;
    if (!empty && a->rot > 0 && (a->pos == nullptr || a->freq == nullptr)) return RED_ERR_INVALID_ARG;
    const bool sums = back && (dqw != nullptr || dkw != nullptr);
    if (empty && !sums) return RED_OK;

    // Elements a lane holds: those of a 16-byte load where every row allows
    // it, 4 elements where 8 bytes (16-bit types) do, else 1 (16384 tokens x 40
    // heads of 128 in bf16, forward / backward: 8 elements 60.8 / 90.9 us, 4
    // elements 65.6 / 117, 1 element 164 / 249).
    auto fits = [&](size_t v) {
        const size_t b = v * es;
        if (D % v != 0 || !rows_on(a->q, T, es, b) || !rows_on(a->k, T, es, b) || !rows_on(a->q_out, T, es, b) ||
            !rows_on(a->k_out, T, es, b) || !is_aligned(a->q_weight, b) || !is_aligned(a->k_weight, b))
            return false;
        return !back || (rows_on(*dq, T, es, b) && rows_on(*dk, T, es, b));
    };
    int vec = (int)(16 / es);
    if (!fits((size_t)vec)) vec = fits(4) ? 4 : 1;
    // Rows that a wave takes at once lie within 2 GiB, else it takes one.
    for (const red_heads* h : {&a->q, &a->k, &a->q_out, &a->k_out, dq, dk})
        if (h != nullptr && h->heads > 1 && h->head_stride > (int64_t)1 << 25) vec = 1;
    int lanes = 4;
    while (lanes < 64 && (size_t)(lanes * vec) < D) lanes *= 2;
    if (vec == 1) lanes = 64;

    int dev, cus;
    red_status st = host_compute_units(&dev, &cus);
    if (st != RED_OK) return st;
    libred::QkNorm k = {};
    k.q = to_heads(a->q), k.k = to_heads(a->k), k.q_out = to_heads(a->q_out), k.k_out = to_heads(a->k_out);
    if (back) k.dq = to_heads(*dq), k.dk = to_heads(*dk);
    k.q_weight = a->q_weight, k.k_weight = a->k_weight;
    k.pos = a->pos, k.freq = a->freq;
    k.tokens = (int64_t)T;
    k.q_heads = (int)a->q.heads, k.k_heads = (int)a->k.heads, k.dim = (int)D;
    k.rot = (int)a->rot, k.interleaved = a->interleaved != 0, k.eps = a->eps;
    // Waves: a token's heads are shared by several where there are few tokens,
    // until there are 4 waves a compute unit or a wave has one pass left (1000
    // tokens x 40 heads, forward / backward: 8.2 / 13.7 us; with 16, where each
    // works out its token's angles for two passes, 10.0 / 17.4; with 2, 9.8 / 15.6).
    const int passes = rows == 0 ? 1 : (rows + 64 / lanes - 1) / (64 / lanes);
    const size_t want = (size_t)cus * 4;
    size_t parts = T >= want || T == 0 ? 1 : (want + T - 1) / T;
    if (parts > (size_t)passes) parts = passes;
    k.parts = (int)parts;
    const size_t items = T * parts;
    size_t blocks = (items + libred::kQkNormWaves - 1) / libred::kQkNormWaves;
    if (blocks == 0) blocks = 1;
    const QkNormLaunch launch = a->type == RED_F32   ? libred::launch_qk_norm_f32
                                : a->type == RED_F16 ? libred::launch_qk_norm_f16
                                                     : libred::launch_qk_norm_bf16;
    if (!back) {
        // Tokens have one wave each where there are so many.
        const size_t most = blocks > kMaxBlocks ? kMaxBlocks * libred::kQkNormWaves : T;
        for (size_t t = 0; t < T; t += most) {
            const size_t n = T - t < most ? T - t : most;
            k.q = heads_from(a->q, t, es), k.k = heads_from(a->k, t, es);
            k.q_out = heads_from(a->q_out, t, es), k.k_out = heads_from(a->k_out, t, es);
            k.pos = a->pos ? a->pos + t : nullptr, k.tokens = (int64_t)n;
            const size_t all = (n * parts + libred::kQkNormWaves - 1) / libred::kQkNormWaves;
            const hipError_t e = launch(vec, lanes, k, false, (int)all, stream);
            if (e != hipSuccess) return host_fail(e, RED_ERR_HIP);
        }
        return RED_OK;
    }
    // Blocks that go through tokens in turn: 6 a compute unit (16384 tokens x
    // 40 heads of 128: 91 us; 5 a compute unit 100, 8 a compute unit 95).
    const size_t cap = (size_t)cus * 6;
    if (blocks > cap) blocks = cap;
    const StreamTurn turn(dev, stream);
    void* partials = nullptr;
    st = host_scratch(dev, stream, blocks * 2 * D * sizeof(float), &partials);
    if (st != RED_OK) return st;
    k.partials = static_cast<float*>(partials);
    hipError_t e = launch(vec, lanes, k, true, (int)blocks, stream);
    if (e == hipSuccess && sums) e = libred::launch_qk_norm_weights(k.partials, (int)blocks, (int)D, dqw, dkw, stream);
    return e == hipSuccess ? RED_OK : host_fail(e, RED_ERR_HIP);
}

red_status cache_call(const red_paged_cache* c, int type, const red_heads* k, const red_heads* v, const int64_t* slots,
                      size_t tokens, bool write, hipStream_t stream) {
    if (!cache_valid(c) || k == nullptr || v == nullptr) return RED_ERR_INVALID_ARG;
    if (type != RED_F16 && type != RED_BF16) return RED_ERR_INVALID_ARG;
    if ((c->type == RED_F16 || c->type == RED_BF16) && c->type != type) return RED_ERR_INVALID_ARG;
    if (tokens > RED_MAX_N) return RED_ERR_INVALID_ARG;
    const size_t D = c->dim;
    for (const red_heads* h : {k, v}) {
        if (h->heads != (int64_t)c->heads || !heads_valid(*h, tokens, D, 2)) return RED_ERR_INVALID_ARG;
        if (!write && !rows_apart(*h, tokens, D)) return RED_ERR_INVALID_ARG;
    }
    if (tokens > 0 && (slots == nullptr || !is_aligned(slots, 8))) return RED_ERR_INVALID_ARG;
    if (tokens == 0 || (write && c->pages == 0)) return RED_OK;
    const size_t cb = type_bytes(c->type);
    // 8 elements a lane, or 1 where rows do not start on 16 bytes (8 in 8 bits;
    // 32768 tokens x 16 rows of 128, e4m3: write / read 44.8 / 36.1 us, with 1
    // element 104 / 64).
    const int vec = D % 8 == 0 && rows_on(*k, tokens, 2, 16) && rows_on(*v, tokens, 2, 16) && cache_rows_on(*c, 8 * cb) ? 8 : 1;
    int lanes = 8;
    while ((size_t)(lanes * vec) < D) lanes *= 2;
    if (vec == 1) lanes = 64;
    int dev, cus;
    const red_status st = host_compute_units(&dev, &cus);
    if (st != RED_OK) return st;
    libred::CacheRows a = {};
    a.cache = to_cache(*c);
    a.k = to_heads(*k), a.v = to_heads(*v);
    a.slots = slots, a.tokens = (int64_t)tokens;
    if (c->pages == 0) {
        // A read of nothing: no slot is inside, but the kernel's loads (of the
        // first row of every head) are made all the same and dropped, so they
        // get memory to read: the outputs' first row and the first slot, for
        // all heads, since the strides of no pages say nothing.
        a.cache.k = k->data, a.cache.v = v->data;
        a.cache.k_scales = a.cache.v_scales = reinterpret_cast<float*>(const_cast<int64_t*>(slots));
        a.cache.head_stride = a.cache.scale_head_stride = 0;
    }
    const size_t block_tokens = (size_t)(libred::kCacheWaves * 64 / lanes);
    const size_t groups = (tokens + block_tokens - 1) / block_tokens;
    // A block takes all heads of its tokens; where that makes too few blocks
    // for 4 a compute unit the heads are shared, down to one row a group (20
    // tokens x 16 rows, write / read: 3.4 / 3.1 us, not shared 9.1 / 5.1; 32768
    // tokens: 44.8 / 36.1, shared 69 / 49).
    const size_t want = (size_t)cus * 4, pairs = 2 * c->heads;
    size_t parts = groups >= want ? 1 : (want + groups - 1) / groups;
    if (parts > pairs) parts = pairs;
    if (parts > 65535) parts = 65535;
    a.parts = (int)parts;
    const size_t most = groups > kMaxBlocks ? kMaxBlocks * block_tokens : tokens;
    for (size_t t = 0; t < tokens; t += most) {
        const size_t n = tokens - t < most ? tokens - t : most;
        a.k = heads_from(*k, t, 2), a.v = heads_from(*v, t, 2);
        a.slots = slots + t, a.tokens = (int64_t)n;
        const unsigned int all = (unsigned int)((n + block_tokens - 1) / block_tokens);
        const hipError_t e = write ? libred::launch_cache_write(type, c->type, vec, lanes, a, all, stream)
                                   : libred::launch_cache_read(type, c->type, vec, lanes, a, all, stream);
        if (e != hipSuccess) return host_fail(e, RED_ERR_HIP);
    }
    return RED_OK;
}

// table_head: from one kv head's table to the next.
red_status attention_call(const red_tree_attention_args* a, int64_t table_head, hipStream_t stream) {
    if (a == nullptr || !cache_valid(&a->cache)) return RED_ERR_INVALID_ARG;
    const red_paged_cache& c = a->cache;
    const int type = a->type;
    if (type != RED_F16 && type != RED_BF16) return RED_ERR_INVALID_ARG;
    if ((c.type == RED_F16 || c.type == RED_BF16) && c.type != type) return RED_ERR_INVALID_ARG;
    const size_t D = c.dim, B = a->batch, N = a->nodes, H = a->q_heads, G = H / c.heads;
    if (D % 16 != 0 || !cache_rows_on(c, 16)) return RED_ERR_INVALID_ARG;
    if (N > RED_TREE_MAX_NODES || H % c.heads != 0 || H > 65535 || B > 65535) return RED_ERR_INVALID_ARG;
    if (a->max_len > (size_t)1 << 30 || a->table_cols > (size_t)1 << 30 || a->table_stride < 0) return RED_ERR_INVALID_ARG;
    if (table_head < 0 || table_head > (int64_t)1 << 40) return RED_ERR_INVALID_ARG;
    if (a->table_stride > (int64_t)1 << 40 || !(a->scale - a->scale == 0.f)) return RED_ERR_INVALID_ARG;
    if (B == 0 || N == 0 || H == 0) return RED_OK;
    if (a->q == nullptr || a->out == nullptr || a->lse == nullptr || a->lens == nullptr) return RED_ERR_INVALID_ARG;
    if (!is_aligned(a->q, 16) || !is_aligned(a->out, 16) || !is_aligned(a->lse, 4) || !is_aligned(a->lens, 4) ||
        !is_aligned(a->table, 4) || !is_aligned(a->tree_mask, 8) || !is_aligned(a->node_count, 4))
        return RED_ERR_INVALID_ARG;
    const size_t tokens = a->table_cols * c.places < a->max_len ? a->table_cols * c.places : a->max_len;
    if (tokens > 0 && a->table == nullptr) return RED_ERR_INVALID_ARG;
    // (batch, node) pairs and heads: rows of q on 16-byte boundaries, rows of
    // out as well and apart from each other.
    // Rows are found by 32-bit numbers of 16 bytes from the head's first.
    const int64_t es = (int64_t)type_bytes(c.type), unit = 16 / es;
    const int64_t rows_span = c.pages == 0 ? 0 : paged_span(c, c.page_stride, 0, c.place_stride, D) / unit;
    if (rows_span > 0xFFFFFFFFll || c.scale_page_stride > 0xFFFFFFFFll || c.scale_place_stride > 0xFFFFFFFFll)
        return RED_ERR_INVALID_ARG;
    const int64_t lim = (int64_t)1 << 40, d = (int64_t)D;
    const int64_t qb = B > 1 ? a->q_batch_stride : 0, qn = N > 1 ? a->q_node_stride : 0, qh = H > 1 ? a->q_head_stride : 0;
    const int64_t bs = B > 1 ? a->out_batch_stride : 0, ns = N > 1 ? a->out_node_stride : 0, hs = H > 1 ? a->out_head_stride : 0;
    for (const int64_t s : {qb, qn, qh, bs, ns, hs})
        if (s < 0 || s > lim || s % 8 != 0) return RED_ERR_INVALID_ARG;
    const int64_t head_span = ((int64_t)H - 1) * hs + d, node_span = ((int64_t)N - 1) * ns + head_span;
    if ((H > 1 && hs < d) || (N > 1 && ns < head_span) || (B > 1 && bs < node_span)) return RED_ERR_INVALID_ARG;
    const red_heads q = {const_cast<void*>(a->q), (int64_t)B, 0, qb};
    const red_heads o = {a->out, (int64_t)B, 0, bs};
    const int64_t q_span = ((int64_t)N - 1) * qn + ((int64_t)H - 1) * qh + d;
    const uintptr_t q0 = (uintptr_t)q.data, qe = q0 + 2 * (uintptr_t)span_of(q, 1, (size_t)q_span);
    const uintptr_t o0 = (uintptr_t)o.data, oe = o0 + 2 * (uintptr_t)span_of(o, 1, (size_t)node_span);
    if (q0 < oe && o0 < qe) return RED_ERR_INVALID_ARG;

    int dev, cus;
    red_status st = host_compute_units(&dev, &cus);
    if (st != RED_OK) return st;
    libred::TreeAttention k = {};
    k.q = a->q, k.out = a->out, k.lse = a->lse;
    k.q_batch = qb, k.q_node = qn, k.q_head = qh;
    k.out_batch = bs, k.out_node = ns, k.out_head = hs;
    k.cache = to_cache(c);
    k.table = a->table, k.table_stride = a->table_stride, k.table_head = table_head;
    k.lens = a->lens, k.mask = a->tree_mask, k.count = a->node_count;
    k.batch = (int)B, k.nodes = (int)N, k.group = (int)G, k.max_tokens = c.pages == 0 ? 0 : (int)tokens;
    k.keep = a->scale == 0.f ? 0u : 0xFFFFFFFFu;
    k.scale = (a->scale == 0.f ? 1.f : a->scale < 0.f ? -a->scale : a->scale) * 1.4426950408889634f;
    k.flip = a->scale < 0.f ? 0x80008000u : 0u;
    k.page16 = (uint32_t)(c.pages > 1 ? c.page_stride / unit : 0), k.place16 = (uint32_t)(c.places > 1 ? c.place_stride / unit : 0);
    while ((size_t)1 << k.places_shift < c.places) ++k.places_shift;
    k.places_factor = (uint32_t)(((uint64_t)1 << (30 + k.places_shift)) / c.places + 1);
    const size_t M = N * G;
    const libred::AttentionShape shape = libred::attention_shape((int)M, (int)D, c.type == RED_F16 || c.type == RED_BF16 ? 2 : 1);
    k.row_blocks = (int)((M + shape.rows() - 1) / shape.rows());
    // As many blocks as the card holds at once, or one a tile; or one a segment,
    // which needs no joining. The cost of the first is the joining: a launch
    // and latency, and the sums written and read. The cost of the second are
    // the turns that its blocks take more (of a wave's 32 tokens, or of a
    // block's 32 or 64), if few: lengths may differ more than the host knows.
    // 4 segments of 2 / 3 / 4 / 8 tiles (us, kernels alone):
    //   shared, 32 rows of 128, int8    14.0   12.6   13.0   13.4
    //   a block a segment               10.8   12.7   14.2   21.2
    // 64 segments of 4 / 6 / 8 tiles of 128 rows of 128, bf16:
    //   shared 24.4   26.3   28.0, a block a segment 16.1   19.5   22.6
    // The constants are fitted to these two rows of shapes; heads above 128 were
    // not among them.
    const size_t tile = (size_t)shape.tokens(), tiles = ((size_t)k.max_tokens + tile - 1) / tile;
    const size_t segments = B * c.heads * (size_t)k.row_blocks;
    if (segments * (tiles > 0 ? tiles : 1) > 0x7fffffff) return RED_ERR_INVALID_ARG;
    const size_t hold = (size_t)cus * (size_t)libred::attention_blocks((int)M, (int)D);
    const size_t blocks = segments * tiles < hold ? segments * tiles : hold;
    std::optional<StreamTurn> turn;  // where there is scratch
    if (k.max_tokens > libred::attention_least_tokens((int)M, (int)D, c.type == RED_F16 || c.type == RED_BF16 ? 2 : 1)) {
        // The scratch is asked for whichever way is taken, and also for one
        // tile where fewer rows would have several, so that a call of a larger
        // shape has always provided that of a smaller one, which a capture
        // relies on.
        const size_t rows = (blocks + segments) * (size_t)shape.rows(), plan = (B + 2 + 3) / 4 * 4;
        turn.emplace(dev, stream);
        void* p = nullptr;
        st = host_scratch(dev, stream, rows * (D * sizeof(float) + sizeof(float2)) + plan * sizeof(int), &p);
        if (st != RED_OK && tiles > 1) return st;  // one tile a segment needs none itself
        const size_t more = tiles * ((segments + hold - 1) / hold) - (segments * tiles + hold - 1) / hold;
        const size_t turn_ns = 7 * D * (size_t)(shape.waves_t > 1 ? 2 : shape.step / 32);
        if (tiles > 8 || more * turn_ns > 5500 + rows * D * sizeof(float) / 2500) {
            k.blocks = (int)blocks;
            k.part_o = static_cast<float*>(p);
            k.part_ml = reinterpret_cast<float2*>(k.part_o + rows * D);
            k.plan = reinterpret_cast<int*>(k.part_ml + rows);
        }
    }
    if (k.blocks > 0) {
        hipError_t e = libred::launch_tree_attention(type, c.type, k, stream);
        if (e == hipSuccess) e = libred::launch_attention_combine(type, k, shape.rows(), stream);
        return e == hipSuccess ? RED_OK : host_fail(e, RED_ERR_HIP);
    }
    // A block a segment: as many sequences a launch as it may have blocks for.
    const size_t most = segments > kMaxBlocks ? kMaxBlocks / (segments / B) : B;
    for (size_t b = 0; b < B; b += most) {
        k.batch = (int)(B - b < most ? B - b : most);
        k.q = static_cast<const char*>(a->q) + (int64_t)b * qb * 2, k.out = static_cast<char*>(a->out) + (int64_t)b * bs * 2;
        k.lse = a->lse + b * N * H;
        k.table = a->table ? a->table + (int64_t)b * a->table_stride : nullptr, k.lens = a->lens + b;
        k.mask = a->tree_mask ? a->tree_mask + b * N : nullptr, k.count = a->node_count ? a->node_count + b : nullptr;
        const hipError_t e = libred::launch_tree_attention(type, c.type, k, stream);
        if (e != hipSuccess) return host_fail(e, RED_ERR_HIP);
    }
    return RED_OK;
}

// Whether batch x steps rows of `vocab` elements at these strides stay in range.
bool rows_in_range(int64_t batch_stride, int64_t step_stride, size_t batch, size_t steps, size_t vocab) {
    const red_heads h = {nullptr, (int64_t)steps, batch_stride, step_stride};
    return span_of(h, batch, vocab) >= 0;
}

red_status verify_call(const red_verify_drafts_args* a, hipStream_t stream) {
    if (a == nullptr) return RED_ERR_INVALID_ARG;
    if (a->type != RED_F32 && a->type != RED_F16 && a->type != RED_BF16) return RED_ERR_INVALID_ARG;
    const size_t es = type_bytes(a->type), B = a->batch, K = a->drafts, V = a->vocab;
    if (B > 65535 || K > 1 << 20 || V < 1 || V > (size_t)1 << 40) return RED_ERR_INVALID_ARG;
    if (B == 0) return RED_OK;
    if (a->p == nullptr || a->r == nullptr || a->accepted == nullptr || a->tokens == nullptr) return RED_ERR_INVALID_ARG;
    if (K > 0 && (a->drafted == nullptr || a->u == nullptr)) return RED_ERR_INVALID_ARG;
    if (!is_aligned(a->p, es) || !is_aligned(a->q, es) || !is_aligned(a->drafted, 8) || !is_aligned(a->u, 4) ||
        !is_aligned(a->r, 4) || !is_aligned(a->draft_count, 4) || !is_aligned(a->accepted, 4) || !is_aligned(a->tokens, 8))
        return RED_ERR_INVALID_ARG;
    if (!rows_in_range(a->p_batch_stride, a->p_step_stride, B, K + 1, V)) return RED_ERR_INVALID_ARG;
    if (a->q != nullptr && !rows_in_range(a->q_batch_stride, a->q_step_stride, B, K, V)) return RED_ERR_INVALID_ARG;
    int dev, cus;
    red_status st = host_compute_units(&dev, &cus);
    if (st != RED_OK) return st;
    libred::Verify k = {};
    k.p = a->p, k.q = a->q;
    k.p_batch = a->p_batch_stride, k.p_step = a->p_step_stride;
    k.q_batch = a->q_batch_stride, k.q_step = a->q_step_stride;
    k.drafted = a->drafted, k.u = a->u, k.r = a->r, k.count = a->draft_count;
    k.accepted = a->accepted, k.tokens = a->tokens;
    k.vocab = (int64_t)V, k.batch = (int)B, k.drafts = (int)K;
    // Segments of 1024 tokens, or as many times that as leave at most 256.
    const size_t least = (V + libred::kVerifyMaxSegs - 1) / libred::kVerifyMaxSegs;
    k.seg = (int64_t)((least + 1023) / 1024 * 1024);
    k.segs = (int)((V + (size_t)k.seg - 1) / (size_t)k.seg);
    // Waves: 32 a compute unit over the batch, each with segments in turn (192
    // rows of 131071: 33 us; 16 and 48 a compute unit 35, a wave a segment 40).
    const size_t waves = ((size_t)cus * 32 + B - 1) / B, all = ((size_t)k.segs + 3) / 4;
    k.blocks = (int)(all < (waves + 3) / 4 ? all : (waves + 3) / 4);
    // One launch, a block of 16 waves a sequence, where that is one turn of them
    // or the sequences fill half of the card and it is a few (float32 rows of
    // 8000 / 32000 / 64000 / 131071; two launches and one, us):
    //   1 sequence      8.1 / 7.4 / 7.6 / 8.4,      7.7 / 9.8 / 14.4 / 26.2
    //   192 sequences   10.6 / 15.8 / 22.0 / 34.1,  9.8 / 13.8 / 20.7 / 37.1
    // More sequences than the card holds such blocks of would take turns.
    if (B <= (size_t)cus * 2 && (k.segs <= 16 || (B >= (size_t)cus / 2 && k.segs <= 64))) k.blocks = 0;
    const StreamTurn turn(dev, stream);
    // The scratch is that of as many segments as a smaller vocabulary may have,
    // and is asked for where one launch keeps its sums in the LDS as well: a
    // call of a larger shape has then always provided that of a smaller one,
    // which a capture relies on.
    const size_t most = (V + 1023) / 1024 < (size_t)libred::kVerifyMaxSegs ? (V + 1023) / 1024 : (size_t)libred::kVerifyMaxSegs;
    void* sums = nullptr;
    st = host_scratch(dev, stream, B * most * sizeof(double), &sums);
    if (st != RED_OK) return st;
    k.sums = static_cast<double*>(sums);
    const hipError_t e = libred::launch_verify(a->type, k, stream);
    return e == hipSuccess ? RED_OK : host_fail(e, RED_ERR_HIP);
}

}  // namespace

extern "C" {

red_status red_qk_norm_rope(const red_qk_norm_rope_args* a, hipStream_t stream) {
    return qk_norm_call(a, nullptr, nullptr, nullptr, nullptr, false, stream);
}

red_status red_qk_norm_rope_backward(const red_qk_norm_rope_args* a, const red_heads* dq, const red_heads* dk,
                                     float* dq_weight, float* dk_weight, hipStream_t stream) {
    return qk_norm_call(a, dq, dk, dq_weight, dk_weight, true, stream);
}

red_status red_cache_write(const red_paged_cache* cache, int type, const red_heads* k, const red_heads* v,
                           const int64_t* slots, size_t tokens, hipStream_t stream) {
    return cache_call(cache, type, k, v, slots, tokens, true, stream);
}

red_status red_cache_read(const red_paged_cache* cache, int type, const red_heads* k, const red_heads* v,
                          const int64_t* slots, size_t tokens, hipStream_t stream) {
    return cache_call(cache, type, k, v, slots, tokens, false, stream);
}

red_status red_tree_attention(const red_tree_attention_args* a, hipStream_t stream) {
    return attention_call(a, 0, stream);
}

red_status red_sparse_attention(const red_tree_attention_args* a, int64_t table_head_stride, hipStream_t stream) {
    return attention_call(a, table_head_stride, stream);
}

red_status red_verify_drafts(const red_verify_drafts_args* a, hipStream_t stream) { return verify_call(a, stream); }

}  // extern "C"
