// serve.cpp -- the C entry points of libred_serve.h: argument checks, launch
// shapes, and the calls into the kernels. (red_sparse_attention is beside
// red_tree_attention, in decode.cpp.)
#include "serve.hpp"

#include <optional>

#include "decode_host.hpp"

using namespace libred;

namespace {

constexpr size_t kMost32 = 0x7fffffff;

// Whether [p, p + bytes) and [q, q + more) meet.
bool meet(const void* p, size_t bytes, const void* q, size_t more) {
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return bytes && more && a < b + more && b < a + bytes;
}

red_status plan_call(const red_plan_slots_args* a, hipStream_t stream) {
    if (a == nullptr) return RED_ERR_INVALID_ARG;
    const size_t B = a->batch, T = a->tokens, C = a->table_cols;
    if (B > 65535 || T > kMost32 || a->pages > kMost32 || C > (size_t)1 << 30 || B * C > kMost32) return RED_ERR_INVALID_ARG;
    if (a->places < 1 || a->places > (size_t)1 << 20 || a->table_stride < 0 || a->table_stride > (int64_t)1 << 40)
        return RED_ERR_INVALID_ARG;
    if (B > 1 && C > 0 && a->table_stride < (int64_t)C) return RED_ERR_INVALID_ARG;  // rows of an output lie apart
    if (a->starts == nullptr || a->free_count == nullptr || (T > 0 && (a->slots == nullptr || a->pos == nullptr))) return RED_ERR_INVALID_ARG;
    if (B > 0 && (a->lens == nullptr || a->counts == nullptr || a->held == nullptr || a->granted == nullptr)) return RED_ERR_INVALID_ARG;
    if ((a->pages > 0 && a->free_pages == nullptr) || (B > 0 && C > 0 && a->table == nullptr)) return RED_ERR_INVALID_ARG;
    for (const void* p : {(const void*)a->lens, (const void*)a->counts, (const void*)a->done, (const void*)a->table, (const void*)a->held,
                          (const void*)a->free_pages, (const void*)a->free_count, (const void*)a->starts, (const void*)a->granted})
        if (!is_aligned(p, 4)) return RED_ERR_INVALID_ARG;
    if (!is_aligned(a->slots, 8) || !is_aligned(a->pos, 8)) return RED_ERR_INVALID_ARG;
    // Nothing that is written lies over anything else.
    struct Span {
        const void* p;
        size_t bytes;
        bool out;
    };
    const Span spans[] = {{a->lens, B * 4, false},
                          {a->counts, B * 4, false},
                          {a->done, a->done ? B * 4 : 0, false},
                          {a->table, B && C ? ((B - 1) * (size_t)a->table_stride + C) * 4 : 0, true},
                          {a->held, B * 4, true},
                          {a->free_pages, a->pages * 4, true},
                          {a->free_count, 4, true},
                          {a->slots, T * 8, true},
                          {a->pos, T * 8, true},
                          {a->starts, (B + 1) * 4, true},
                          {a->granted, B * 4, true}};
    for (const Span& x : spans)
        for (const Span& y : spans)
            if (&x != &y && x.out && meet(x.p, x.bytes, y.p, y.bytes)) return RED_ERR_INVALID_ARG;
    int dev, cus;
    red_status st = host_compute_units(&dev, &cus);
    if (st != RED_OK) return st;
    const StreamTurn turn(dev, stream);
    void* p = nullptr;
    st = host_scratch(dev, stream, (3 * (B + 1) + 4 + a->pages) * sizeof(int32_t), &p);
    if (st != RED_OK) return st;
    PlanSlots k = {};
    k.lens = a->lens, k.counts = a->counts, k.done = a->done;
    k.table = a->table, k.table_stride = a->table_stride;
    k.held = a->held, k.stack = a->free_pages, k.height = a->free_count;
    k.slots = a->slots, k.pos = a->pos, k.starts = a->starts, k.granted = a->granted;
    k.batch = (int)B, k.tokens = (int)T, k.cols = (int)C, k.places = (int)a->places, k.pages = (int)a->pages;
    k.have = static_cast<int32_t*>(p);
    k.before = k.have + B + 1, k.back = k.before + B + 1, k.sums = k.back + B + 1, k.fresh = k.sums + 4;
    const size_t wide = (T + 255) / 256 < (size_t)cus * 8 ? (T + 255) / 256 : (size_t)cus * 8;
    // One block, or the tokens in a launch of their own. (Microseconds, replayed:
    // 1024 tokens 7.4 / 8.8, 4096 tokens 12.6 / 10.2, 16384 tokens 34 / 12.)
    const int blocks = T <= 2048 ? 0 : (int)wide;
    // The block of the sums moves the pages too, if few are taken, else a launch of
    // its own does. (Replayed: 256 pages 10.2 / 11.5, 1024 pages 11.6 / 12.9, 2048
    // pages 14.4 / 14.3, 16384 pages 43 / 14; from Python, where a launch more is 2 us
    // of the host's, 2100 taken and 16000 given back 15.4 / 17.3.) Neither rule knows the
    // pages given back, whose number is on the device: 256 rows that end at once take one
    // block 46 us with 64 pages each, 164 with 256, 650 with 1024 and 10.5 ms with 16384.
    const bool few = T / a->places + B <= 4096;
    const hipError_t e = launch_plan_slots(k, blocks, few, stream);
    return e == hipSuccess ? RED_OK : host_fail(e, RED_ERR_HIP);
}

// Whether rows of bounds of these strides can be read 16 bytes at a time.
bool bounds_on_16(const void* lo, const void* hi, int64_t page_stride, int64_t head_stride, size_t pages, size_t heads) {
    return is_aligned(lo, 16) && is_aligned(hi, 16) && (pages <= 1 || page_stride % 8 == 0) && (heads == 1 || head_stride % 8 == 0);
}

// Elements spanned by the bounds, -1 if out of range.
int64_t bounds_span(int64_t page_stride, int64_t head_stride, size_t pages, size_t heads, size_t dim) {
    const red_heads h = {nullptr, (int64_t)heads, page_stride, head_stride};
    return span_of(h, pages, dim);
}

int row_lanes(size_t dim, int vec) {
    int lanes = 8;
    while ((size_t)(lanes * vec) < dim) lanes *= 2;
    return vec == 1 ? 64 : lanes;
}

red_status bounds_call(const red_page_bounds_args* a, hipStream_t stream) {
    if (a == nullptr) return RED_ERR_INVALID_ARG;
    red_paged_cache c = a->cache;
    const bool scaled = c.type == RED_I8 || c.type == RED_E4M3;
    c.v = c.k, c.v_scales = c.k_scales;  // the values are not read
    if (!cache_valid(&c)) return RED_ERR_INVALID_ARG;
    if (a->type != RED_F16 && a->type != RED_BF16) return RED_ERR_INVALID_ARG;
    if (!scaled && c.type != a->type) return RED_ERR_INVALID_ARG;
    const size_t B = a->batch, D = c.dim, H = c.heads;
    if (B > 65535 || a->table_cols > (size_t)1 << 30 || a->table_stride < 0 || a->table_stride > (int64_t)1 << 40) return RED_ERR_INVALID_ARG;
    const size_t most = a->most < a->table_cols ? a->most : a->table_cols;
    if (a->bound_page_stride < 0 || a->bound_head_stride < 0) return RED_ERR_INVALID_ARG;
    if (B == 0 || most == 0 || c.pages == 0) return RED_OK;
    if (a->lo == nullptr || a->hi == nullptr || a->table == nullptr || a->lens == nullptr) return RED_ERR_INVALID_ARG;
    if (!is_aligned(a->lo, 2) || !is_aligned(a->hi, 2) || !is_aligned(a->table, 4) || !is_aligned(a->lens, 4) || !is_aligned(a->first, 4))
        return RED_ERR_INVALID_ARG;
    const red_heads rows = {a->lo, (int64_t)H, a->bound_page_stride, a->bound_head_stride};
    const int64_t span = bounds_span(a->bound_page_stride, a->bound_head_stride, c.pages, H, D);
    if (span < 0 || !rows_apart(rows, c.pages, D)) return RED_ERR_INVALID_ARG;
    const size_t bytes = (size_t)span * 2, keys = (size_t)paged_span(c, c.page_stride, c.head_stride, c.place_stride, D) * type_bytes(c.type);
    if (meet(a->lo, bytes, a->hi, bytes) || meet(a->lo, bytes, c.k, keys) || meet(a->hi, bytes, c.k, keys)) return RED_ERR_INVALID_ARG;
    PageBounds k = {};
    k.cache = to_cache(c);
    k.table = a->table, k.table_stride = a->table_stride, k.lens = a->lens, k.first = a->first;
    k.lo = a->lo, k.hi = a->hi, k.bound_page = a->bound_page_stride, k.bound_head = a->bound_head_stride;
    k.cols = (int)a->table_cols, k.most = (int)most;
    const size_t blocks = (most * H + kBoundsWaves - 1) / kBoundsWaves;
    if (blocks > kMaxBlocks) return RED_ERR_INVALID_ARG;
    int dev, cus;
    const red_status st = host_compute_units(&dev, &cus);
    if (st != RED_OK) return st;
    const size_t cb = type_bytes(c.type);
    const int load = (int)(16 / cb);  // elements
    const int vec = D % load == 0 && cache_rows_on(c, 16) && bounds_on_16(a->lo, a->hi, a->bound_page_stride, a->bound_head_stride, c.pages, H) ? load : 1;
    const size_t each = kMaxBlocks / blocks < B ? kMaxBlocks / blocks : B;  // sequences a launch
    for (size_t b = 0; b < B; b += each) {
        k.table = a->table + (int64_t)b * a->table_stride, k.lens = a->lens + b, k.first = a->first ? a->first + b : nullptr;
        const hipError_t e = launch_page_bounds(a->type, c.type, vec, row_lanes(D, vec), k, (unsigned)blocks,
                                                (unsigned)(B - b < each ? B - b : each), stream);
        if (e != hipSuccess) return host_fail(e, RED_ERR_HIP);
    }
    return RED_OK;
}

red_status select_call(const red_select_pages_args* a, hipStream_t stream) {
    if (a == nullptr || (a->type != RED_F16 && a->type != RED_BF16)) return RED_ERR_INVALID_ARG;
    const size_t B = a->batch, N = a->nodes, H = a->kv_heads, D = a->dim;
    if (B > 65535 || N > RED_TREE_MAX_NODES || H < 1 || a->q_heads < 1 || a->q_heads > 65535 || a->q_heads % H != 0) return RED_ERR_INVALID_ARG;
    if (D < 1 || D > RED_HEAD_MAX_DIM || a->places < 1 || a->places > (size_t)1 << 20 || a->pages > kMost32) return RED_ERR_INVALID_ARG;
    if (a->max_len > (size_t)1 << 30 || a->table_cols > (size_t)1 << 30 || a->table_stride < 0 || a->table_stride > (int64_t)1 << 40)
        return RED_ERR_INVALID_ARG;
    if (a->budget < 1 || a->budget > (size_t)1 << 30 || a->first > a->budget || a->last > a->budget) return RED_ERR_INVALID_ARG;
    if (a->first + a->last + 1 + (N + a->places - 1) / a->places > a->budget) return RED_ERR_INVALID_ARG;
    if (a->q_batch_stride < 0 || a->q_node_stride < 0 || a->q_head_stride < 0) return RED_ERR_INVALID_ARG;
    const int64_t lim = (int64_t)1 << 40;
    if (a->q_batch_stride > lim || a->q_node_stride > lim || a->q_head_stride > lim) return RED_ERR_INVALID_ARG;
    const int64_t span = a->pages == 0 ? 0 : bounds_span(a->bound_page_stride, a->bound_head_stride, a->pages, H, D);
    if (span < 0) return RED_ERR_INVALID_ARG;
    if (B == 0) return RED_OK;
    if (a->selected == nullptr || a->selected_lens == nullptr || a->lens == nullptr) return RED_ERR_INVALID_ARG;
    const size_t tokens = a->table_cols * a->places < a->max_len ? a->table_cols * a->places : a->max_len;
    const size_t most = (tokens + a->places - 1) / a->places;
    if (most > 0 && a->table == nullptr) return RED_ERR_INVALID_ARG;
    const bool scored = most > a->budget && N > 0;
    if (scored && (a->q == nullptr || (a->pages > 0 && (a->lo == nullptr || a->hi == nullptr)))) return RED_ERR_INVALID_ARG;
    if (!is_aligned(a->q, 2) || !is_aligned(a->lo, 2) || !is_aligned(a->hi, 2)) return RED_ERR_INVALID_ARG;
    for (const void* p : {(const void*)a->table, (const void*)a->lens, (const void*)a->node_count, (const void*)a->selected, (const void*)a->selected_lens})
        if (!is_aligned(p, 4)) return RED_ERR_INVALID_ARG;
    if (B * H > kMost32 / a->budget || (most > 0 && B * H > kMost32 / most)) return RED_ERR_INVALID_ARG;
    // The outputs lie over none of the small inputs (those of q and the bounds
    // are other types' tensors).
    const size_t out = B * H * a->budget * 4, table = B && most ? ((B - 1) * (size_t)a->table_stride + a->table_cols) * 4 : 0;
    for (const void* p : {(const void*)a->selected, (const void*)a->selected_lens}) {
        const size_t bytes = p == a->selected ? out : B * 4;
        if (meet(p, bytes, a->table, table) || meet(p, bytes, a->lens, B * 4) || meet(p, bytes, a->node_count, a->node_count ? B * 4 : 0))
            return RED_ERR_INVALID_ARG;
    }
    if (meet(a->selected, out, a->selected_lens, B * 4)) return RED_ERR_INVALID_ARG;
    int dev, cus;
    red_status st = host_compute_units(&dev, &cus);
    if (st != RED_OK) return st;
    // A block that scores pages first adds up the queries: 64 pages of it, or as
    // many times that as leave 4 blocks a compute unit.
    const size_t parts = B * H * ((most + kSelectPages - 1) / kSelectPages) / ((size_t)cus * 4);
    const size_t share = kSelectPages * (parts < 1 ? 1 : parts);
    const size_t blocks = H * ((most + share - 1) / share);  // a sequence; few thousand a kv head at most
    SelectPages k = {};
    k.q = a->q, k.q_batch = a->q_batch_stride, k.q_node = a->q_node_stride, k.q_head = a->q_head_stride;
    k.lo = a->lo, k.hi = a->hi, k.bound_page = a->bound_page_stride, k.bound_head = a->bound_head_stride;
    k.table_stride = a->table_stride, k.pages = (int64_t)a->pages;
    k.nodes = (int)N, k.heads = (int)H, k.group = (int)(a->q_heads / H), k.dim = (int)D, k.places = (int)a->places;
    k.budget = (int)a->budget, k.first = (int)a->first, k.last = (int)a->last;
    k.most = (int)most, k.share = (int)share, k.max_len = (int)tokens;
    const StreamTurn turn(dev, stream);
    // Asked for where the budget takes all pages as well, so that a call provides
    // it for those of a smaller budget.
    void* p = nullptr;
    if (most > 0) {
        st = host_scratch(dev, stream, B * H * most * sizeof(uint64_t), &p);
        if (st != RED_OK) return st;
    }
    // Bounds 16 bytes at a time, and queries 8.
    const bool q_on_8 = is_aligned(a->q, 8) && (B == 1 || a->q_batch_stride % 4 == 0) && (N <= 1 || a->q_node_stride % 4 == 0) &&
                        (a->q_heads == 1 || a->q_head_stride % 4 == 0);
    const int vec = D % 8 == 0 && q_on_8 && bounds_on_16(a->lo, a->hi, a->bound_page_stride, a->bound_head_stride, a->pages, H) ? 8 : 1;
    // A launch has fewer than 2^32 threads; those that choose come in 1024 at most.
    const size_t most_blocks = blocks > H * 4 ? kMaxBlocks / blocks : kMaxBlocks / (4 * H);
    const size_t each = most_blocks < B ? most_blocks : B;
    for (size_t b = 0; b < B; b += each) {
        k.batch = (int)(B - b < each ? B - b : each);
        k.q = a->q ? static_cast<const char*>(a->q) + (int64_t)b * a->q_batch_stride * 2 : nullptr;
        k.table = a->table ? a->table + (int64_t)b * a->table_stride : nullptr;
        k.lens = a->lens + b, k.count = a->node_count ? a->node_count + b : nullptr;
        k.selected = a->selected + b * H * a->budget, k.selected_lens = a->selected_lens + b;
        k.keys = static_cast<uint64_t*>(p);
        const hipError_t e = launch_select_pages(a->type, vec, row_lanes(D, vec), k, stream);
        if (e != hipSuccess) return host_fail(e, RED_ERR_HIP);
    }
    return RED_OK;
}

bool float_type(int type) { return type == RED_F32 || type == RED_F16 || type == RED_BF16; }

red_status sample_call(const red_sample_args* a, hipStream_t stream) {
    if (a == nullptr || !float_type(a->type)) return RED_ERR_INVALID_ARG;
    const size_t B = a->batch, S = a->steps, V = a->vocab, es = type_bytes(a->type);
    if (B > 65535 || S > 65535 || B * S >= (size_t)1 << 22 || V < 1 || V > (size_t)1 << 20) return RED_ERR_INVALID_ARG;
    if (B == 0 || S == 0) return RED_OK;
    if (a->logits == nullptr || !is_aligned(a->logits, es) || (a->tokens != nullptr && a->r == nullptr)) return RED_ERR_INVALID_ARG;
    for (const void* p : {(const void*)a->temperature, (const void*)a->top_k, (const void*)a->top_p, (const void*)a->min_p, (const void*)a->r})
        if (!is_aligned(p, 4)) return RED_ERR_INVALID_ARG;
    if (!is_aligned(a->tokens, 8)) return RED_ERR_INVALID_ARG;
    const red_heads x = {const_cast<void*>(a->logits), (int64_t)S, a->batch_stride, a->step_stride};
    const int64_t span = span_of(x, B, V);
    if (span < 0 || meet(a->tokens, a->tokens ? B * S * 8 : 0, a->logits, (size_t)span * es)) return RED_ERR_INVALID_ARG;
    if (a->probs != nullptr) {
        const size_t ps = float_type(a->probs_type) ? type_bytes(a->probs_type) : 0;
        const red_heads p = {a->probs, (int64_t)S, a->probs_batch_stride, a->probs_step_stride};
        if (ps == 0 || !is_aligned(a->probs, ps) || span_of(p, B, V) < 0 || !rows_apart(p, B, V)) return RED_ERR_INVALID_ARG;
        const size_t bytes = (size_t)span_of(p, B, V) * ps;
        if (meet(a->probs, bytes, a->logits, (size_t)span * es) || meet(a->probs, bytes, a->tokens, a->tokens ? B * S * 8 : 0)) return RED_ERR_INVALID_ARG;
    }
    if (a->tokens == nullptr && a->probs == nullptr) return RED_OK;
    int dev, cus;
    red_status st = host_compute_units(&dev, &cus);
    if (st != RED_OK) return st;
    Sample k = {};
    k.x = a->logits, k.batch_stride = a->batch_stride, k.step_stride = a->step_stride;
    k.temperature = a->temperature, k.top_k = a->top_k, k.top_p = a->top_p, k.min_p = a->min_p, k.r = a->r;
    k.tokens = a->tokens, k.probs = a->probs, k.probs_batch = a->probs_batch_stride, k.probs_step = a->probs_step_stride;
    k.steps = (int)S, k.vocab = (int)V;
    // The sum of all weights stays below 2^62, one weight below 2^52.
    int log2 = 0;
    while ((size_t)1 << log2 < V) ++log2;
    k.shift = 62 - log2 < 51 ? 62 - log2 : 51;
    k.filtered = a->top_k != nullptr || a->top_p != nullptr || a->min_p != nullptr;
    const int probs_type = a->probs != nullptr ? a->probs_type : RED_F32;
    const size_t rows = B * S;
    size_t each = rows;
    std::optional<StreamTurn> turn;  // where there is scratch
    if (V > kSampleRow) {
        turn.emplace(dev, stream);
        // Rows cut into chunks, as many at a time as 256 MiB hold the bins and
        // lists of.
        const size_t chunks = (V + kSampleChunk - 1) / kSampleChunk;
        const size_t row = chunks * (sizeof(SampleHead) + kSampleGrid * 8) + kSampleList * 8 + sizeof(SamplePlan);
        constexpr size_t most = (size_t)256 << 20;
        void* p = nullptr;
        st = host_scratch(dev, stream, rows < most / row ? rows * row : most, &p);
        if (st != RED_OK) return st;
        if (each > most / row) each = most / row;
        k.chunks = (int)chunks;
        k.bins = static_cast<unsigned long long*>(p);
        k.list = k.bins + each * chunks * kSampleGrid;
        k.heads = reinterpret_cast<SampleHead*>(k.list + each * kSampleList);
        k.plans = reinterpret_cast<SamplePlan*>(k.heads + each * chunks);
    }
    for (size_t at = 0; at < rows; at += each) {
        k.first_row = (int)at;
        const hipError_t e = launch_sample(a->type, probs_type, k, (unsigned)(rows - at < each ? rows - at : each), stream);
        if (e != hipSuccess) return host_fail(e, RED_ERR_HIP);
    }
    return RED_OK;
}

}  // namespace

extern "C" {

red_status red_plan_slots(const red_plan_slots_args* a, hipStream_t stream) { return plan_call(a, stream); }

red_status red_page_bounds(const red_page_bounds_args* a, hipStream_t stream) { return bounds_call(a, stream); }

red_status red_select_pages(const red_select_pages_args* a, hipStream_t stream) { return select_call(a, stream); }

red_status red_sample(const red_sample_args* a, hipStream_t stream) { return sample_call(a, stream); }

}  // extern "C"
