// kvattend_abi.cpp - the C ABI of the operators of kvattend.h: host-side
// validation, size queries and kernel launches.
//
// As in kvcodec_abi.cpp, nothing here touches the GPU except the launch calls.
#include "kvattend.h"

#include <math.h>

#include <initializer_list>
#include <numeric>

#include "attend.h"
#include "layout.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
    if (na == 0 || nb == 0) return false;
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + nb && y < x + na;
}

// A set of head vectors: n tokens x heads x d channels. Strides of counts of
// 1 are taken as those of packed rows.
struct View {
    const void* data;
    uint64_t ts, hs;  // elements
    uint64_t n, heads, d;
    uint64_t bytes;   // from the first to behind the last element
};

// Strides fit, and the range of bytes they span stays below 2^62.
bool view_of(const kvc_rows* r, uint64_t n, uint64_t heads, uint64_t d, View& v) {
    v = View{r->data, r->token_stride, r->head_stride, n, heads, d, 0};
    if (heads == 1) v.hs = d;
    if (n == 1) v.ts = heads * d;
    const unsigned __int128 last = (unsigned __int128)(n - 1) * v.ts + (unsigned __int128)(heads - 1) * v.hs + d;
    if (last >= ((unsigned __int128)1 << 61)) return false;
    v.bytes = (uint64_t)last * 2;
    return true;
}

bool view_aligned(const View& v) { return aligned(v.data, 16) && v.ts % 8 == 0 && v.hs % 8 == 0; }

// Whether no two of its vectors share an element.
bool view_apart(const View& v) {
    const unsigned __int128 row = (unsigned __int128)(v.heads - 1) * v.hs + v.d;   // one token's heads
    const unsigned __int128 plane = (unsigned __int128)(v.n - 1) * v.ts + v.d;     // one head's tokens
    const bool heads_inside = v.hs >= v.d && (v.n == 1 || v.ts >= row);
    const bool tokens_inside = v.ts >= v.d && (v.heads == 1 || v.hs >= plane);
    return heads_inside || tokens_inside;
}

// Whether two sets of vectors may share an element: their ranges meet, and no stride S tells them apart, that
// is, modulo S all of the one lies in places of its own. S is tried as the token stride of both (each token's
// heads together, as the rows of one buffer), the head stride of both (each head's tokens together), and the
// greatest common divisor of all strides (single vectors, as of [tokens][heads][3][d]).
bool views_meet(const View& a, const View& b) {
    if (!overlap(a.data, a.bytes, b.data, b.bytes)) return false;
    const View& x = (uintptr_t)a.data <= (uintptr_t)b.data ? a : b;
    const View& y = (uintptr_t)a.data <= (uintptr_t)b.data ? b : a;
    const uint64_t apart = (uintptr_t)y.data - (uintptr_t)x.data;
    // elements that x and y take from their place on, of every S
    const auto told_apart = [&](uint64_t S, unsigned __int128 ex, unsigned __int128 ey) {
        if (ex > S || ey > S) return false;
        const uint64_t off = apart % (2 * S);
        return off >= 2 * ex && 2 * S - off >= 2 * ey;
    };
    const auto together = [](uint64_t count, uint64_t stride, uint64_t d) {
        return (unsigned __int128)(count - 1) * stride + d;
    };
    if (x.n > 1 && y.n > 1 && x.ts == y.ts && told_apart(x.ts, together(x.heads, x.hs, x.d), together(y.heads, y.hs, y.d)))
        return false;
    if (x.heads > 1 && y.heads > 1 && x.hs == y.hs && told_apart(x.hs, together(x.n, x.ts, x.d), together(y.n, y.ts, y.d)))
        return false;
    uint64_t g = 0;
    for (const View* v : {&x, &y}) {
        if (v->n > 1) g = std::gcd(g, v->ts);
        if (v->heads > 1) g = std::gcd(g, v->hs);
    }
    return !told_apart(g, x.d, y.d);
}

bool view_meets(const View& a, const void* p, uint64_t n) { return overlap(a.data, a.bytes, p, n); }

bool same_view(const View& a, const View& b) { return a.data == b.data && a.ts == b.ts && a.hs == b.hs; }

kvc::RowsDev rows_dev(const View& v) {
    return kvc::RowsDev{static_cast<uint16_t*>(const_cast<void*>(v.data)), v.ts, v.hs};
}

bool spec_ok(const kvc_pages* s) {
    if (!s || !kvc::page_spec_ok(s->num_pages, s->num_kv_heads, s->page_tokens, s->head_dim, s->format)) return false;
    // all byte offsets below 2^62
    const kvc::PageLayout l = kvc::page_layout(1, s->num_kv_heads, s->page_tokens, s->head_dim, s->format);
    return (unsigned __int128)l.page_bytes * s->num_pages < ((unsigned __int128)1 << 62);
}

kvc::PageLayout layout_of(const kvc_pages* s) {
    return kvc::page_layout(s->num_pages, s->num_kv_heads, s->page_tokens, s->head_dim, s->format);
}

int page_copy(bool write, const kvc_pages* spec, const void* pages, size_t pages_bytes, uint32_t n, const kvc_rows* k,
              const kvc_rows* v, const int64_t* slots, int32_t* dev_status, hipStream_t stream) {
    if (!spec) return KVC_E_NULL;
    if (!spec_ok(spec) || n >= (1u << 26)) return KVC_E_SHAPE;
    if (n == 0) return KVC_OK;
    if (!pages || !k || !v || !k->data || !v->data || !slots) return KVC_E_NULL;
    const kvc::PageLayout lay = layout_of(spec);
    const uint64_t need = lay.page_bytes * lay.num_pages;
    if (pages_bytes < need) return KVC_E_SIZE;
    View kv, vv;
    if (!view_of(k, n, lay.H, lay.d, kv) || !view_of(v, n, lay.H, lay.d, vv)) return KVC_E_SHAPE;
    if (!aligned(pages, 256) || !view_aligned(kv) || !view_aligned(vv) || !aligned(slots, 8) ||
        (dev_status && !aligned(dev_status, 4)))
        return KVC_E_ALIGN;
    const uint64_t sb = (uint64_t)n * 8, tb = dev_status ? 4 : 0;
    if (view_meets(kv, pages, need) || view_meets(vv, pages, need) || overlap(pages, need, dev_status, tb) ||
        overlap(slots, sb, dev_status, tb) || view_meets(kv, dev_status, tb) || view_meets(vv, dev_status, tb))
        return KVC_E_ALIAS;
    if (write) {
        if (overlap(pages, need, slots, sb)) return KVC_E_ALIAS;
    } else if (!view_apart(kv) || !view_apart(vv) || views_meet(kv, vv) || view_meets(kv, slots, sb) ||
               view_meets(vv, slots, sb)) {
        return KVC_E_ALIAS;
    }
    const hipError_t e = write ? kvc::launch_page_write(lay, const_cast<void*>(pages), n, rows_dev(kv), rows_dev(vv), slots,
                                                        dev_status, stream)
                               : kvc::launch_page_read(lay, pages, n, slots, rows_dev(kv), rows_dev(vv), dev_status, stream);
    return e == hipSuccess ? KVC_OK : KVC_E_HIP;
}

// query rows: a launch has fewer than 2^32 threads, 256 for each row at most
bool heads_ok(uint64_t n, uint32_t H, uint32_t Hq) {
    return H >= 1 && Hq >= 1 && Hq % H == 0 && Hq <= (1u << 16) && n * Hq < (1ull << 23);
}
// tokens of all sequences, in the 128-token blocks that the kernels count
bool tokens_ok(uint64_t n, uint64_t max_tokens) { return max_tokens < (1ull << 31) && n * (max_tokens / 128 + 1) < (1ull << 31); }
bool plan_ok(const kvc::AttendPlan& p) {
    return p.units < (1ull << 23) && p.slots < (1ull << 31) && p.blocks < (1ull << 40);
}

// Checks of a page source; `most`: table_cols * page_tokens.
int check_tail(const kvc_pages* spec, const void* pages, size_t pages_bytes, uint32_t n, const int32_t* table,
               uint32_t table_cols, uint64_t table_stride, const int32_t* lens) {
    if (!spec) return KVC_E_NULL;
    if (!spec_ok(spec)) return KVC_E_SHAPE;
    if (!pages || !table || !lens) return KVC_E_NULL;
    if (table_cols < 1 || (uint64_t)table_cols * spec->page_tokens >= (1ull << 31)) return KVC_E_SHAPE;
    if (table_stride >= (1ull << 31) || (n > 1 && table_stride < table_cols && table_stride != 0)) return KVC_E_RANGE;
    if (pages_bytes < kvpage_bytes(spec)) return KVC_E_SIZE;
    if (!aligned(pages, 256) || !aligned(table, 4) || !aligned(lens, 4)) return KVC_E_ALIGN;
    return KVC_OK;
}

// finite, and so in powers of two
bool scale_ok(float scale) { return isfinite(scale * 1.4426950408889634f); }

struct Span {
    const void* p;
    uint64_t n;
};

// Whether rows or spans that are written meet what else a call reads or writes.
template <int I, int O>
bool spans_meet(const View& q, const View& out, const Span (&ins)[I], const Span (&outs)[O]) {
    for (const Span& x : ins)
        if (view_meets(out, x.p, x.n)) return true;
    for (int i = 0; i < O; ++i) {
        if (view_meets(out, outs[i].p, outs[i].n) || view_meets(q, outs[i].p, outs[i].n)) return true;
        for (const Span& x : ins)
            if (overlap(outs[i].p, outs[i].n, x.p, x.n)) return true;
        for (int j = i + 1; j < O; ++j)
            if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return true;
    }
    return false;
}

// Workspace bytes of a call: `need`, what it uses, and `room`, which serves every smaller call too; false
// if an argument is invalid.
struct Workspace {
    uint64_t need, room;
    bool add(const kvc::AttendPlan& p, uint32_t d) {
        need += p.bytes(d);
        room += p.room;
        return plan_ok(p);
    }
};
bool page_workspace(const kvc_pages* spec, uint32_t n, uint32_t q_heads, uint32_t max_tokens, uint32_t window,
                    uint32_t sinks, Workspace& w) {
    w = Workspace{0, 0};
    if (!spec_ok(spec) || !heads_ok(n, spec->num_kv_heads, q_heads) || !tokens_ok(n, max_tokens)) return false;
    if (n == 0) w = Workspace{256, 256};
    const uint32_t d = spec->head_dim;
    const uint64_t most = kvc::seen_tokens(max_tokens, window, sinks);
    return n == 0 || w.add(kvc::page_attend_plan(n, spec->num_kv_heads, q_heads, d, most, false), d);
}
bool pool_workspace(const kvc_shape* s, uint32_t n, uint32_t q_heads, const kvc_pages* tail, uint32_t max_tokens,
                    Workspace& w) {
    w = Workspace{0, 0};
    if (!s || !kvc::pool_shape_ok(s->num_layers, s->num_kv_heads, s->num_tokens, s->head_dim) ||
        !heads_ok(n, s->num_kv_heads, q_heads))
        return false;
    if (tail && (!spec_ok(tail) || tail->num_kv_heads != s->num_kv_heads || tail->head_dim != s->head_dim ||
                 !tokens_ok(n, max_tokens)))
        return false;
    if (n == 0) {
        w = Workspace{256, 256};
        return true;
    }
    const uint32_t H = s->num_kv_heads, d = s->head_dim;
    const kvc::AttendPlan p = kvc::pool_attend_plan(H, n, q_heads, d, s->num_tokens, tail != nullptr);
    if (!w.add(p, d)) return false;
    if (!tail) return true;
    const kvc::AttendPlan t = kvc::page_attend_plan(n, H, q_heads, d, max_tokens, true);
    return w.add(t, d) && t.W + p.W < (1ull << 31);
}

bool rotation_ok(uint32_t head_dim, float eps, uint32_t n_pairs, uint32_t pairing) {
    return pairing <= 1 && n_pairs % 8 == 0 && n_pairs <= head_dim / 2 && eps >= 0.0f && !isinf(eps);
}

// The window and the sinks of a call: no window where it holds every token that a table's row can; sinks up to those.
void take_window(kvc::TailArgs& t, uint32_t window, uint32_t sinks) {
    const uint32_t most = t.table_cols * t.lay.P;
    t.window = window < most ? window : 0;
    t.sinks = sinks < most ? sinks : most;
}

// kvpage_attend, with a window (0: none) and sinks
int attend_pages(const kvc_pages* spec, const void* pages, size_t pages_bytes, uint32_t n_seqs, uint32_t q_heads,
                 const kvc_rows* q, const int32_t* table, uint32_t table_cols, uint64_t table_stride,
                 const int32_t* lens, uint32_t window, uint32_t sinks, float scale, const kvc_rows* out, float* lse,
                 void* ws, size_t ws_bytes, int32_t* dev_status, hipStream_t stream) {
    if (!spec) return KVC_E_NULL;
    if (!spec_ok(spec) || !heads_ok(n_seqs, spec->num_kv_heads, q_heads)) return KVC_E_SHAPE;
    if (!scale_ok(scale)) return KVC_E_RANGE;
    if (n_seqs == 0) return KVC_OK;
    if (!q || !out || !q->data || !out->data || !ws) return KVC_E_NULL;
    const int rc = check_tail(spec, pages, pages_bytes, n_seqs, table, table_cols, table_stride, lens);
    if (rc != KVC_OK) return rc;
    Workspace w;
    if (!page_workspace(spec, n_seqs, q_heads, table_cols * spec->page_tokens, window, sinks, w)) return KVC_E_SHAPE;
    const uint64_t need = w.need;
    if (ws_bytes < need) return KVC_E_SIZE;
    View qv, ov;
    if (!view_of(q, n_seqs, q_heads, spec->head_dim, qv) || !view_of(out, n_seqs, q_heads, spec->head_dim, ov))
        return KVC_E_SHAPE;
    if (!view_aligned(qv) || !view_aligned(ov) || !aligned(ws, 256) || (lse && !aligned(lse, 4)) ||
        (dev_status && !aligned(dev_status, 4)))
        return KVC_E_ALIGN;
    const Span ins[3] = {{pages, kvpage_bytes(spec)},
                         {table, ((uint64_t)(n_seqs - 1) * table_stride + table_cols) * 4},
                         {lens, (uint64_t)n_seqs * 4}};
    const Span outs[3] = {{lse, lse ? (uint64_t)n_seqs * q_heads * 4 : 0}, {ws, need}, {dev_status, dev_status ? 4u : 0u}};
    if (!view_apart(ov) || views_meet(ov, qv) || spans_meet(qv, ov, ins, outs)) return KVC_E_ALIAS;
    kvc::AttendArgs a{};
    a.n = n_seqs;
    a.H = spec->num_kv_heads;
    a.Hq = q_heads;
    a.d = spec->head_dim;
    a.q = rows_dev(qv);
    a.out = rows_dev(ov);
    a.scale = scale;
    a.lse = lse;
    a.ws = ws;
    a.status = dev_status;
    a.tail = kvc::TailArgs{layout_of(spec), static_cast<const uint8_t*>(pages), table, table_cols, table_stride, lens,
                           0, 0};
    take_window(a.tail, window, sinks);
    return kvc::launch_attend(a, stream) == hipSuccess ? KVC_OK : KVC_E_HIP;
}

// What kvpage_attend_prompt takes, before its pages are looked at.
bool prompt_ok(const kvc_pages* s, uint64_t n_seqs, uint64_t n_tokens, uint32_t q_heads) {
    if (!spec_ok(s)) return false;
    const uint64_t H = s->num_kv_heads;
    return q_heads >= 1 && q_heads % H == 0 && q_heads <= (1u << 16) && n_tokens * q_heads < (1ull << 30) &&
           n_seqs < (1u << 20) && H * (n_tokens * (q_heads / H) / kvc::kPromptRows + n_seqs) < (1ull << 23);
}

}  // namespace

extern "C" {

int kvc_norm_rotate(uint32_t n_tokens, uint32_t q_heads, uint32_t kv_heads, uint32_t head_dim, const kvc_rows* q_in,
                    const kvc_rows* k_in, const void* q_weight, const void* k_weight, float eps,
                    const int64_t* positions, const float* inv_freq, uint32_t n_pairs, uint32_t pairing,
                    const kvc_rows* q_out, const kvc_rows* k_out, hipStream_t stream) {
    // four tokens a workgroup of 256 threads, fewer than 2^32 threads a launch
    if ((head_dim != 64 && head_dim != 128) || q_heads > (1u << 16) || kv_heads > (1u << 16) ||
        n_tokens > (1u << 26) - 4)
        return KVC_E_SHAPE;
    if (!rotation_ok(head_dim, eps, n_pairs, pairing)) return KVC_E_RANGE;
    if (n_tokens == 0 || q_heads + kv_heads == 0) return KVC_OK;
    if (n_pairs && (!positions || !inv_freq)) return KVC_E_NULL;
    const kvc_rows* ins[2] = {q_in, k_in};
    const kvc_rows* outs[2] = {q_out, k_out};
    const uint32_t heads[2] = {q_heads, kv_heads};
    const void* weights[2] = {q_weight, k_weight};
    for (int i = 0; i < 2; ++i)
        if (heads[i] && (!ins[i] || !outs[i] || !ins[i]->data || !outs[i]->data)) return KVC_E_NULL;
    View vi[2]{}, vo[2]{};
    for (int i = 0; i < 2; ++i)
        if (heads[i] && (!view_of(ins[i], n_tokens, heads[i], head_dim, vi[i]) ||
                         !view_of(outs[i], n_tokens, heads[i], head_dim, vo[i])))
            return KVC_E_SHAPE;
    for (int i = 0; i < 2; ++i)
        if (heads[i] && (!view_aligned(vi[i]) || !view_aligned(vo[i]) || (weights[i] && !aligned(weights[i], 16))))
            return KVC_E_ALIGN;
    if (n_pairs && !aligned(positions, 8)) return KVC_E_ALIGN;
    for (int i = 0; i < 2; ++i) {
        if (!heads[i]) continue;
        if (!view_apart(vo[i])) return KVC_E_ALIAS;
        for (int j = 0; j < 2; ++j) {
            if (!heads[j]) continue;
            if (!(i == j && same_view(vo[i], vi[j])) && views_meet(vo[i], vi[j])) return KVC_E_ALIAS;
            if (j > i && views_meet(vo[i], vo[j])) return KVC_E_ALIAS;
            if (weights[j] && view_meets(vo[i], weights[j], head_dim * 2)) return KVC_E_ALIAS;
        }
        if (n_pairs && view_meets(vo[i], positions, (uint64_t)n_tokens * 8)) return KVC_E_ALIAS;
    }
    kvc::RotateArgs a{};
    a.n = n_tokens;
    a.Hq = q_heads;
    a.Hk = kv_heads;
    a.d = head_dim;
    a.q_in = rows_dev(vi[0]);
    a.k_in = rows_dev(vi[1]);
    a.q_out = rows_dev(vo[0]);
    a.k_out = rows_dev(vo[1]);
    // (weights without heads are not checked, and kernels load what they are given)
    a.q_weight = q_heads ? q_weight : nullptr;
    a.k_weight = kv_heads ? k_weight : nullptr;
    a.eps = eps;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.n_pairs = n_pairs;
    a.pairing = pairing;
    return kvc::launch_norm_rotate(a, stream) == hipSuccess ? KVC_OK : KVC_E_HIP;
}

size_t kvpage_bytes(const kvc_pages* spec) {
    if (!spec_ok(spec)) return 0;
    const kvc::PageLayout l = layout_of(spec);
    return (size_t)(l.page_bytes * l.num_pages);
}

int kvpage_write(const kvc_pages* spec, void* pages, size_t pages_bytes, uint32_t n_tokens, const kvc_rows* k,
                 const kvc_rows* v, const int64_t* slots, int32_t* dev_status, hipStream_t stream) {
    return page_copy(true, spec, pages, pages_bytes, n_tokens, k, v, slots, dev_status, stream);
}

int kvpage_read(const kvc_pages* spec, const void* pages, size_t pages_bytes, uint32_t n_tokens, const int64_t* slots,
                const kvc_rows* k_out, const kvc_rows* v_out, int32_t* dev_status, hipStream_t stream) {
    return page_copy(false, spec, pages, pages_bytes, n_tokens, k_out, v_out, slots, dev_status, stream);
}

int kvpage_append(const kvc_pages* spec, void* pages, size_t pages_bytes, uint32_t n_tokens, uint32_t q_heads,
                  const kvc_rows* q_in, const kvc_rows* k_in, const kvc_rows* v_in, const void* q_weight,
                  const void* k_weight, float eps, const int64_t* positions, const float* inv_freq, uint32_t n_pairs,
                  uint32_t pairing, const int64_t* slots, const kvc_rows* q_out, int32_t* dev_status,
                  hipStream_t stream) {
    if (!spec) return KVC_E_NULL;
    // four tokens a workgroup of 256 threads, fewer than 2^32 threads a launch
    if (!spec_ok(spec) || q_heads > (1u << 16) || n_tokens > (1u << 26) - 4) return KVC_E_SHAPE;
    const uint32_t d = spec->head_dim, H = spec->num_kv_heads;
    if (!rotation_ok(d, eps, n_pairs, pairing)) return KVC_E_RANGE;
    if (n_tokens == 0) return KVC_OK;
    if (!pages || !k_in || !v_in || !k_in->data || !v_in->data || !slots || (n_pairs && (!positions || !inv_freq)))
        return KVC_E_NULL;
    if (q_heads && (!q_in || !q_out || !q_in->data || !q_out->data)) return KVC_E_NULL;
    const kvc::PageLayout lay = layout_of(spec);
    const uint64_t need = lay.page_bytes * lay.num_pages;
    if (pages_bytes < need) return KVC_E_SIZE;
    View in[3]{}, out{};  // queries, keys, values
    if (!view_of(k_in, n_tokens, H, d, in[1]) || !view_of(v_in, n_tokens, H, d, in[2]) ||
        (q_heads && (!view_of(q_in, n_tokens, q_heads, d, in[0]) || !view_of(q_out, n_tokens, q_heads, d, out))))
        return KVC_E_SHAPE;
    if (!aligned(pages, 256) || !view_aligned(in[1]) || !view_aligned(in[2]) || !aligned(slots, 8) ||
        (n_pairs && !aligned(positions, 8)) || (q_heads && (!view_aligned(in[0]) || !view_aligned(out))) ||
        (q_heads && q_weight && !aligned(q_weight, 16)) || (k_weight && !aligned(k_weight, 16)) ||
        (dev_status && !aligned(dev_status, 4)))
        return KVC_E_ALIGN;
    const Span ins[4] = {{positions, n_pairs ? (uint64_t)n_tokens * 8 : 0},
                         {slots, (uint64_t)n_tokens * 8},
                         {q_weight, q_heads && q_weight ? d * 2u : 0u},
                         {k_weight, k_weight ? d * 2u : 0u}};
    const Span outs[2] = {{pages, need}, {dev_status, dev_status ? 4u : 0u}};
    for (int i = q_heads ? 0 : 1; i < 3; ++i) {
        if (view_meets(in[i], outs[0].p, outs[0].n) || view_meets(in[i], outs[1].p, outs[1].n)) return KVC_E_ALIAS;
        if (q_heads && !(i == 0 && same_view(out, in[0])) && views_meet(out, in[i])) return KVC_E_ALIAS;
    }
    // (without queries `out` is empty and meets nothing)
    if ((q_heads && !view_apart(out)) || spans_meet(in[1], out, ins, outs)) return KVC_E_ALIAS;
    kvc::AppendArgs a{};
    a.n = n_tokens;
    a.Hq = q_heads;
    a.lay = lay;
    a.pages = static_cast<uint8_t*>(pages);
    a.q_in = rows_dev(in[0]);
    a.k_in = rows_dev(in[1]);
    a.v_in = rows_dev(in[2]);
    a.q_out = rows_dev(out);
    a.q_weight = q_heads ? q_weight : nullptr;  // (as above)
    a.k_weight = k_weight;
    a.eps = eps;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.n_pairs = n_pairs;
    a.pairing = pairing;
    a.slots = slots;
    a.status = dev_status;
    return kvc::launch_append(a, stream) == hipSuccess ? KVC_OK : KVC_E_HIP;
}

size_t kvpage_attend_workspace_bytes(const kvc_pages* spec, uint32_t n_seqs, uint32_t q_heads, uint32_t max_tokens) {
    Workspace w;
    return page_workspace(spec, n_seqs, q_heads, max_tokens, 0, 0, w) ? (size_t)w.room : 0;
}

int kvpage_attend(const kvc_pages* spec, const void* pages, size_t pages_bytes, uint32_t n_seqs, uint32_t q_heads,
                  const kvc_rows* q, const int32_t* table, uint32_t table_cols, uint64_t table_stride,
                  const int32_t* lens, float scale, const kvc_rows* out, float* lse, void* ws, size_t ws_bytes,
                  int32_t* dev_status, hipStream_t stream) {
    return attend_pages(spec, pages, pages_bytes, n_seqs, q_heads, q, table, table_cols, table_stride, lens, 0, 0, scale,
                        out, lse, ws, ws_bytes, dev_status, stream);
}

size_t kvpage_attend_window_workspace_bytes(const kvc_pages* spec, uint32_t n_seqs, uint32_t q_heads,
                                            uint32_t max_tokens, uint32_t window, uint32_t sinks) {
    Workspace w;
    return page_workspace(spec, n_seqs, q_heads, max_tokens, window, sinks, w) ? (size_t)w.room : 0;
}

int kvpage_attend_window(const kvc_pages* spec, const void* pages, size_t pages_bytes, uint32_t n_seqs,
                         uint32_t q_heads, const kvc_rows* q, const int32_t* table, uint32_t table_cols,
                         uint64_t table_stride, const int32_t* lens, uint32_t window, uint32_t sinks, float scale,
                         const kvc_rows* out, float* lse, void* ws, size_t ws_bytes, int32_t* dev_status,
                         hipStream_t stream) {
    return attend_pages(spec, pages, pages_bytes, n_seqs, q_heads, q, table, table_cols, table_stride, lens, window, sinks,
                        scale, out, lse, ws, ws_bytes, dev_status, stream);
}

size_t kvpage_attend_prompt_workspace_bytes(const kvc_pages* spec, uint32_t n_seqs, uint32_t n_tokens,
                                            uint32_t q_heads, uint32_t max_tokens, uint32_t window, uint32_t sinks) {
    if (!prompt_ok(spec, n_seqs, n_tokens, q_heads) || max_tokens >= (1u << 31)) return 0;
    return (size_t)kvc::prompt_plan(n_seqs, n_tokens, spec->num_kv_heads, q_heads, spec->head_dim, max_tokens, window,
                                    sinks).room;
}

int kvpage_attend_prompt(const kvc_pages* spec, const void* pages, size_t pages_bytes, uint32_t n_seqs,
                         uint32_t n_tokens, uint32_t q_heads, const kvc_rows* q, const int32_t* starts,
                         const int32_t* table, uint32_t table_cols, uint64_t table_stride, const int32_t* lens,
                         uint32_t window, uint32_t sinks, float scale, const kvc_rows* out, float* lse, void* ws,
                         size_t ws_bytes, int32_t* dev_status, hipStream_t stream) {
    if (!spec) return KVC_E_NULL;
    if (!prompt_ok(spec, n_seqs, n_tokens, q_heads)) return KVC_E_SHAPE;
    if (!scale_ok(scale)) return KVC_E_RANGE;
    if (n_seqs == 0 || n_tokens == 0) return KVC_OK;
    if (!q || !out || !q->data || !out->data || !starts || !ws) return KVC_E_NULL;
    const int rc = check_tail(spec, pages, pages_bytes, n_seqs, table, table_cols, table_stride, lens);
    if (rc != KVC_OK) return rc;
    const uint32_t d = spec->head_dim;
    const kvc::PromptPlan plan = kvc::prompt_plan(n_seqs, n_tokens, spec->num_kv_heads, q_heads, d,
                                                  (uint64_t)table_cols * spec->page_tokens, window, sinks);
    if (ws_bytes < plan.bytes) return KVC_E_SIZE;
    View qv, ov;
    if (!view_of(q, n_tokens, q_heads, d, qv) || !view_of(out, n_tokens, q_heads, d, ov)) return KVC_E_SHAPE;
    if (!view_aligned(qv) || !view_aligned(ov) || !aligned(starts, 4) || !aligned(ws, 256) || (lse && !aligned(lse, 4)) ||
        (dev_status && !aligned(dev_status, 4)))
        return KVC_E_ALIGN;
    const Span ins[4] = {{pages, kvpage_bytes(spec)},
                         {table, ((uint64_t)(n_seqs - 1) * table_stride + table_cols) * 4},
                         {lens, (uint64_t)n_seqs * 4},
                         {starts, (uint64_t)n_seqs * 4 + 4}};
    const Span outs[3] = {{lse, lse ? (uint64_t)n_tokens * q_heads * 4 : 0},
                          {ws, plan.bytes},
                          {dev_status, dev_status ? 4u : 0u}};
    if (!view_apart(ov) || views_meet(ov, qv) || spans_meet(qv, ov, ins, outs)) return KVC_E_ALIAS;
    kvc::PromptArgs a{};
    a.n = n_seqs;
    a.rows = n_tokens;
    a.H = spec->num_kv_heads;
    a.Hq = q_heads;
    a.d = d;
    a.q = rows_dev(qv);
    a.out = rows_dev(ov);
    a.scale = scale;
    a.lse = lse;
    a.ws = ws;
    a.status = dev_status;
    a.starts = starts;
    a.tail = kvc::TailArgs{layout_of(spec), static_cast<const uint8_t*>(pages), table, table_cols, table_stride, lens,
                           0, 0};
    take_window(a.tail, window, sinks);
    return kvc::launch_attend_prompt(a, plan, stream) == hipSuccess ? KVC_OK : KVC_E_HIP;
}

size_t kvpool_attend_workspace_bytes(const kvc_shape* shape, uint32_t n_agents, uint32_t q_heads,
                                     const kvc_pages* tail_spec, uint32_t max_tail_tokens) {
    Workspace w;
    return pool_workspace(shape, n_agents, q_heads, tail_spec, max_tail_tokens, w) ? (size_t)w.room : 0;
}

int kvpool_attend(const kvc_shape* shape, const void* pool, size_t pool_bytes, uint32_t layer, uint32_t n_agents,
                  uint32_t q_heads, const kvc_rows* q, float scale, const kvc_tail* tail, const kvc_rows* out,
                  float* lse, void* ws, size_t ws_bytes, int32_t* dev_status, hipStream_t stream) {
    if (!shape) return KVC_E_NULL;
    if (!kvc::pool_shape_ok(shape->num_layers, shape->num_kv_heads, shape->num_tokens, shape->head_dim) ||
        !heads_ok(n_agents, shape->num_kv_heads, q_heads))
        return KVC_E_SHAPE;
    if (layer >= shape->num_layers || !scale_ok(scale)) return KVC_E_RANGE;
    if (n_agents == 0) return KVC_OK;
    if (!pool || !q || !out || !q->data || !out->data || !ws) return KVC_E_NULL;
    const uint32_t H = shape->num_kv_heads, d = shape->head_dim;
    if (tail) {
        const int rc = check_tail(tail->spec, tail->pages, tail->pages_bytes, n_agents, tail->table, tail->table_cols,
                                  tail->table_stride, tail->lens);
        if (rc != KVC_OK) return rc;
        if (tail->spec->num_kv_heads != H || tail->spec->head_dim != d) return KVC_E_SHAPE;
    }
    const uint64_t pool_need = kvpool_bytes(shape);
    Workspace w;
    if (!pool_workspace(shape, n_agents, q_heads, tail ? tail->spec : nullptr,
                        tail ? tail->table_cols * tail->spec->page_tokens : 0, w))
        return KVC_E_SHAPE;
    const uint64_t need = w.need;
    if (pool_bytes < pool_need || ws_bytes < need) return KVC_E_SIZE;
    View qv, ov;
    if (!view_of(q, n_agents, q_heads, d, qv) || !view_of(out, n_agents, q_heads, d, ov)) return KVC_E_SHAPE;
    if (!aligned(pool, 256) || !view_aligned(qv) || !view_aligned(ov) || !aligned(ws, 256) ||
        (lse && !aligned(lse, 4)) || (dev_status && !aligned(dev_status, 4)))
        return KVC_E_ALIGN;
    const Span ins[4] = {
        {pool, pool_need},
        {tail ? tail->pages : nullptr, tail ? kvpage_bytes(tail->spec) : 0},
        {tail ? tail->table : nullptr, tail ? ((uint64_t)(n_agents - 1) * tail->table_stride + tail->table_cols) * 4 : 0},
        {tail ? tail->lens : nullptr, tail ? (uint64_t)n_agents * 4 : 0}};
    const Span outs[3] = {{lse, lse ? (uint64_t)n_agents * q_heads * 4 : 0}, {ws, need}, {dev_status, dev_status ? 4u : 0u}};
    if (!view_apart(ov) || views_meet(ov, qv) || spans_meet(qv, ov, ins, outs)) return KVC_E_ALIAS;
    kvc::AttendArgs a{};
    a.n = n_agents;
    a.H = H;
    a.Hq = q_heads;
    a.d = d;
    a.q = rows_dev(qv);
    a.out = rows_dev(ov);
    a.scale = scale;
    a.lse = lse;
    a.ws = ws;
    a.status = dev_status;
    a.pool = static_cast<const uint8_t*>(pool);
    a.L = shape->num_layers;
    a.T = shape->num_tokens;
    a.layer = layer;
    if (tail)
        a.tail = kvc::TailArgs{layout_of(tail->spec), static_cast<const uint8_t*>(tail->pages), tail->table,
                               tail->table_cols, tail->table_stride, tail->lens, 0, 0};
    return kvc::launch_attend(a, stream) == hipSuccess ? KVC_OK : KVC_E_HIP;
}

}  // extern "C"
