// gdn_attn_api.cpp -- the C ABI's entry points of the softmax attention layer: rotary positions, attention over prompts
// and in decode steps, and the pages of their cache (declared in include/gdn.h).
//
// As in gdn_api.cpp every argument is checked on the host before the first HIP call.

#include "gdn.h"

#include <algorithm>
#include <cmath>

#include "gdn_attn.h"
#include "gdn_checks.h"

namespace {

using namespace gdn::checks;

constexpr int64_t kMaxStride = (int64_t)1 << 24;   // a tile's rows are addressed with 32-bit byte offsets
constexpr int64_t kMaxKeys = (int64_t)1 << 30;     // of a sequence in a decode step, split into runs of at most kMostKeys
constexpr int64_t kMaxPages = (int64_t)1 << 30;    // of a pool, and entries of its table
constexpr int64_t kMaxBlocks = (int64_t)1 << 24;   // a launch holds fewer than 2^32 threads, 256 of them a workgroup

// log2 of a page size that is built, -1 of others
int page_shift_of(int32_t page_size)
{
    for (int shift = 4; shift <= 10; ++shift)
        if (page_size == 1 << shift)
            return shift;
    return -1;
}

// Checks what the attention entry points share, for `rows` queries; fills the kernels' part.
gdn_status check_attention(const gdn_attention_args *a, int64_t rows, gdn::AttnParams &p)
{
    if (!a)
        return GDN_ERR_NULL;
    if (a->q_heads < 1 || a->kv_heads < 1 || a->q_heads % a->kv_heads != 0 || a->page_size < 0 || a->num_pages < 0)
        return GDN_ERR_SHAPE;
    if (!gdn::attn_supported(a->head_dim) || (a->dtype != GDN_F16 && a->dtype != GDN_BF16) ||
        (a->page_size > 0 && page_shift_of(a->page_size) < 0))
        return GDN_ERR_UNSUPPORTED;
    if (!std::isfinite(a->scale) || a->scale < 0.f)
        return GDN_ERR_SHAPE;
    const int64_t q_width = (int64_t)a->q_heads * a->head_dim, k_width = (int64_t)a->kv_heads * a->head_dim;
    if (q_width >= kMaxStride || rows * a->q_heads > kI32Max)
        return GDN_ERR_OVERFLOW;
    p.Hq = a->q_heads;
    p.Hkv = a->kv_heads;
    p.D = a->head_dim;
    p.dt = a->dtype;
    p.scale = a->scale > 0.f ? a->scale : 1.0f / std::sqrt((float)a->head_dim);
    if (rows == 0)
        return GDN_OK;
    if (!a->q || !a->out)
        return GDN_ERR_NULL;
    const int64_t k_least = a->page_size > 0 ? k_width * a->page_size : k_width;
    if (a->q_stride < q_width || a->out_stride < q_width || a->k_stride < k_least || a->v_stride < k_least ||
        (a->page_size > 0 && a->table_stride < 0))
        return GDN_ERR_SHAPE;
    if (a->q_stride >= kMaxStride || a->out_stride >= kMaxStride ||
        (a->page_size == 0 && (a->k_stride >= kMaxStride || a->v_stride >= kMaxStride)))
        return GDN_ERR_OVERFLOW;
    if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || a->q_stride % 8 != 0 ||
        a->out_stride % 8 != 0 || a->k_stride % 8 != 0 || a->v_stride % 8 != 0 || !aligned(a->lse, 4) || !aligned(a->table, 4))
        return GDN_ERR_ALIGN;
    p.q = a->q;
    p.q_stride = a->q_stride;
    p.out = a->out;
    p.out_stride = a->out_stride;
    p.lse = a->lse;
    p.kv.k = a->k;
    p.kv.v = a->v;
    p.kv.k_stride = a->k_stride;
    p.kv.v_stride = a->v_stride;
    p.kv.page_shift = a->page_size > 0 ? page_shift_of(a->page_size) : -1;
    p.kv.num_pages = a->num_pages;
    p.kv.table = a->table;
    p.kv.table_stride = a->table_stride;
    return GDN_OK;
}

bool heads_ok(int32_t q_heads, int32_t kv_heads, int32_t head_dim)
{
    return q_heads >= 1 && kv_heads >= 1 && q_heads % kv_heads == 0 && gdn::attn_supported(head_dim);
}

// Workspace of `rows` rows (queries times heads) of `slots` partial results each: (maximum, sum) pairs, then outputs
size_t stat_bytes(int64_t rows, int64_t slots)
{
    return ((size_t)(rows * slots) * sizeof(float2) + 255) / 256 * 256;
}
size_t split_bytes(int64_t rows, int64_t slots, int D)
{
    return slots <= 1 ? 0 : stat_bytes(rows, slots) + (size_t)(rows * slots) * D * sizeof(float);
}
void carve(gdn::AttnParams &p, int64_t rows, int slots, void *workspace)
{
    p.slots = slots > 1 ? slots : 0;
    p.stat = static_cast<float2 *>(workspace);
    p.part = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + stat_bytes(rows, slots));
}

// How a decode step is split: runs of the prefix's keys, then of each sequence's own
struct DecodeSplit {
    int prefix, prefix_tiles, own, own_keys;
};
DecodeSplit decode_split(int Hq, int Hkv, int D, int B, int T, int max_len, int prefix_len)
{
    DecodeSplit s{};
    if (prefix_len > 0)
        gdn::attn_prefill_splits(Hq, Hkv, D, 1, (int64_t)B * T, nullptr, nullptr, prefix_len, &s.prefix, &s.prefix_tiles);
    gdn::attn_decode_splits(Hq, Hkv, D, B, T, max_len, &s.own, &s.own_keys);
    return s;
}

// Checks the tables that the page operators share.
gdn_status check_pages(const gdn_page_args *a, bool data, gdn::PageParams &p)
{
    if (!a)
        return GDN_ERR_NULL;
    if (a->rows < 0 || a->width < 0 || a->num_pages < 0 || a->table_stride < a->width)
        return GDN_ERR_SHAPE;
    // walked with 32-bit indices, and steps past the last
    if (a->num_pages > kMaxPages || a->width > kMaxPages || (int64_t)a->rows * a->width > kMaxPages)
        return GDN_ERR_OVERFLOW;
    if ((a->rows > 0 && a->width > 0 && !a->table) || (a->num_pages > 0 && !a->refs))
        return GDN_ERR_NULL;
    if (!aligned(a->table, 4) || !aligned(a->refs, 4))
        return GDN_ERR_ALIGN;
    if (data) {
        if (a->num_planes < 0 || a->page_bytes < 0 || a->page_stride < a->page_bytes || a->plane_stride < 0)
            return GDN_ERR_SHAPE;
        if (a->page_bytes > (int64_t)1 << 30 || (int64_t)a->num_planes * a->num_pages > (int64_t)1 << 40)
            return GDN_ERR_OVERFLOW;
        if (a->num_planes > 0 && a->num_pages > 0 && a->page_bytes > 0 && !a->data)
            return GDN_ERR_NULL;
        if (!aligned(a->data, 16) || a->page_bytes % 16 != 0 || a->page_stride % 16 != 0 || a->plane_stride % 16 != 0)
            return GDN_ERR_ALIGN;
        p.data = static_cast<unsigned char *>(a->data);
        p.num_planes = a->num_planes;
        p.plane_stride = a->plane_stride;
        p.page_stride = a->page_stride;
        p.page_bytes = a->page_bytes;
    }
    p.table = a->table;
    p.table_stride = a->table_stride;
    p.rows = a->rows;
    p.width = a->width;
    p.refs = a->refs;
    p.num_pages = a->num_pages;
    p.page_size = a->page_size;
    return GDN_OK;
}

gdn_status check_requests(int32_t n)
{
    return n < 0 ? GDN_ERR_SHAPE : n > gdn::kPageRequests ? GDN_ERR_OVERFLOW : GDN_OK;
}

gdn_status check_page_workspace(const gdn_page_args *a, void *workspace, size_t bytes)
{
    if (!workspace || bytes < gdn::pages_workspace_bytes(a->num_pages))
        return GDN_ERR_WORKSPACE;
    return aligned(workspace, 256) ? GDN_OK : GDN_ERR_ALIGN;
}

}  // namespace

extern "C" {

gdn_status gdn_rope(const gdn_rope_args *a, void *stream)
{
    if (!a)
        return GDN_ERR_NULL;
    if (a->tokens < 0 || a->q_heads < 0 || a->kv_heads < 0 || !std::isfinite(a->magnitude))
        return GDN_ERR_SHAPE;
    if (!dtype_ok(a->dtype) || (a->layout != GDN_ROPE_HALF && a->layout != GDN_ROPE_INTERLEAVED) || a->head_dim < 2 ||
        a->head_dim > 1024 || a->rotary_dim < 2 || a->rotary_dim > a->head_dim || a->rotary_dim % 2 != 0)
        return GDN_ERR_UNSUPPORTED;
    const bool pages = a->k_pages || a->v_pages;
    if (pages && page_shift_of(a->page_size) < 0)
        return GDN_ERR_UNSUPPORTED;
    const int64_t q_width = (int64_t)a->q_heads * a->head_dim, k_width = (int64_t)a->kv_heads * a->head_dim;
    if (q_width >= kMaxStride || k_width >= kMaxStride)
        return GDN_ERR_OVERFLOW;
    if (pages && (a->num_pages < 0 || (int64_t)a->num_pages * a->page_size > kI32Max))
        return a->num_pages < 0 ? GDN_ERR_SHAPE : GDN_ERR_OVERFLOW;
    if (a->tokens == 0)
        return GDN_OK;
    if (!a->positions || !a->inv_freq || (a->q != nullptr) != (a->q_out != nullptr) || (!a->q && !a->k) ||
        (pages && (!a->k || !a->v || !a->k_pages || !a->v_pages || !a->slots)) || (!pages && (a->k != nullptr) != (a->k_out != nullptr)))
        return GDN_ERR_NULL;
    // v goes to pages or nowhere, k to one of the two
    if ((!pages && a->v) || (pages && a->k_out))
        return GDN_ERR_SHAPE;
    if ((a->q && (a->q_heads < 1 || a->q_stride < q_width || a->q_out_stride < q_width)) ||
        (a->k && (a->kv_heads < 1 || a->k_stride < k_width || (!pages && a->k_out_stride < k_width))) ||
        (pages && (a->v_stride < k_width || a->page_stride < k_width * a->page_size)))
        return GDN_ERR_SHAPE;
    const int64_t es = dtype_size(a->dtype);
    if (!aligned(a->positions, 4) || !aligned(a->inv_freq, 8) || !aligned(a->slots, 4) || !aligned(a->q, es) || !aligned(a->k, es) ||
        !aligned(a->v, es) || !aligned(a->q_out, es) || !aligned(a->k_out, es) || !aligned(a->k_pages, es) || !aligned(a->v_pages, es))
        return GDN_ERR_ALIGN;
    if (a->tokens >= kMaxBlocks)
        return GDN_ERR_OVERFLOW;
    gdn::RopeParams p{};
    p.tokens = a->tokens;
    p.Hq = a->q ? a->q_heads : 0;
    p.Hkv = a->k ? a->kv_heads : 0;
    p.D = a->head_dim;
    p.rot = a->rotary_dim;
    p.layout = a->layout;
    p.dt = a->dtype;
    p.magnitude = a->magnitude != 0.f ? a->magnitude : 1.f;
    p.positions = a->positions;
    p.w = a->inv_freq;
    p.q = a->q;
    p.k = a->k;
    p.v = a->v;
    p.q_stride = a->q_stride;
    p.k_stride = a->k_stride;
    p.v_stride = a->v_stride;
    p.q_out = a->q_out;
    p.k_out = a->k_out;
    p.q_out_stride = a->q_out_stride;
    p.k_out_stride = a->k_out_stride;
    if (pages) {
        p.k_pages = a->k_pages;
        p.v_pages = a->v_pages;
        p.page_stride = a->page_stride;
        p.page_shift = page_shift_of(a->page_size);
        p.num_slots = (int64_t)a->num_pages * a->page_size;
        p.slots = a->slots;
    }
    return launch_status(gdn::launch_rope(p, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_rope_frequencies(int32_t rotary_dim, double theta, int32_t scaling, double factor, double original_length,
                                double beta_fast, double beta_slow, double *inv_freq, float *magnitude)
{
    if (!inv_freq || !magnitude)
        return GDN_ERR_NULL;
    if (scaling < GDN_ROPE_PLAIN || scaling > GDN_ROPE_BANDS || rotary_dim < 2 || rotary_dim > 1024 || rotary_dim % 2 != 0 ||
        (scaling == GDN_ROPE_BASE && rotary_dim < 4))
        return GDN_ERR_UNSUPPORTED;
    const auto finite_from = [](double x, double least) { return std::isfinite(x) && x >= least; };
    if (!std::isfinite(theta) || theta <= 1.0 || (scaling != GDN_ROPE_PLAIN && !finite_from(factor, 1.0)))
        return GDN_ERR_SHAPE;
    if (scaling == GDN_ROPE_BANDS &&
        (!finite_from(original_length, 1.0) || !std::isfinite(beta_fast) || !(beta_slow > 0.0) || !(beta_slow <= beta_fast)))
        return GDN_ERR_SHAPE;
    const double r = rotary_dim;
    if (scaling == GDN_ROPE_BASE)
        theta *= std::pow(factor, r / (r - 2));
    // index of the pair that turns `times` times in original_length tokens
    const auto index_of = [&](double times) {
        return r * std::log(original_length / (times * 2.0 * 3.14159265358979323846)) / (2.0 * std::log(theta));
    };
    double low = 0, high = 0;
    if (scaling == GDN_ROPE_BANDS) {
        low = std::clamp(std::floor(index_of(beta_fast)), 0.0, r - 1);
        high = std::clamp(std::ceil(index_of(beta_slow)), 0.0, r - 1);
    }
    for (int32_t i = 0; i < rotary_dim / 2; ++i) {
        const double w = std::pow(theta, -2.0 * i / r);
        double slow = 0;  // share of w / factor
        if (scaling == GDN_ROPE_LINEAR)
            slow = 1;
        else if (scaling == GDN_ROPE_BANDS)
            slow = high > low ? std::clamp((i - low) / (high - low), 0.0, 1.0) : (i > low ? 1.0 : 0.0);
        inv_freq[i] = slow == 0 ? w : w * (1 - slow) + w / factor * slow;
    }
    *magnitude = scaling == GDN_ROPE_BANDS ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
    return GDN_OK;
}

size_t gdn_attention_prefill_workspace_bytes(int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t num_seqs,
                                             int32_t total_tokens)
{
    if (!heads_ok(q_heads, kv_heads, head_dim) || num_seqs < 0 || total_tokens < 1)
        return 0;
    return split_bytes((int64_t)total_tokens * q_heads, gdn::attn_prefill_most_splits(q_heads, kv_heads, total_tokens), head_dim);
}

gdn_status gdn_attention_prefill(const gdn_attention_args *args, int32_t num_seqs, const int32_t *cu_q_host,
                                 const int32_t *cu_q_dev, const int32_t *cu_k_host, const int32_t *cu_k_dev, void *workspace,
                                 size_t workspace_bytes, void *stream)
{
    gdn::AttnPrefillParams p{};
    if (num_seqs < 0)
        return GDN_ERR_SHAPE;
    if (!args || !cu_q_host || !cu_q_dev || (cu_k_host != nullptr) != (cu_k_dev != nullptr))
        return GDN_ERR_NULL;
    if (!cu_k_host) {
        cu_k_host = cu_q_host;
        cu_k_dev = cu_q_dev;
    }
    const int32_t total = cu_q_host[num_seqs];
    int64_t sum = 0, longest = 0, longest_k = 0;
    gdn_status st = check_cu(cu_q_host, num_seqs, total, 1, &sum, &longest);
    if (st == GDN_OK)
        st = check_cu(cu_k_host, num_seqs, cu_k_host[num_seqs], 1, &sum, &longest_k);
    if (st == GDN_OK)
        st = check_attention(args, total, p.a);
    if (st != GDN_OK || total == 0)
        return st;
    if (longest_k > 0 && (!args->k || !args->v || (args->page_size > 0 && !args->table)))
        return GDN_ERR_NULL;
    if (args->page_size > 0 && longest_k > 0 && (args->num_pages < 1 || args->table_stride < (longest_k + args->page_size - 1) / args->page_size))
        return GDN_ERR_SHAPE;
    if (longest_k > gdn::kMostKeys)
        return GDN_ERR_OVERFLOW;
    p.N = num_seqs;
    p.total = total;
    p.cu_q = cu_q_dev;
    p.cu_k = cu_k_dev;
    gdn::attn_prefill_splits(p.a.Hq, p.a.Hkv, p.a.D, num_seqs, total, cu_q_host, cu_k_host, 0, &p.splits, &p.split_tiles);
    if (gdn::attn_prefill_blocks(p.a.Hq, p.a.Hkv, num_seqs, total, true) * p.splits >= kMaxBlocks)
        return GDN_ERR_OVERFLOW;
    const int64_t rows = (int64_t)total * p.a.Hq;
    // of the size that the query gives, also where these sequences are too short to be split
    const size_t need = gdn_attention_prefill_workspace_bytes(p.a.Hq, p.a.Hkv, p.a.D, num_seqs, total);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return GDN_ERR_WORKSPACE;
    if (!aligned(workspace, 256))
        return GDN_ERR_ALIGN;
    carve(p.a, rows, p.splits, workspace);
    p.whole = true;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = gdn::launch_attn_prefill(p, s);
    if (e == hipSuccess && p.a.slots > 0)
        e = gdn::launch_attn_join(p.a, rows, s);
    return launch_status(e);
}

size_t gdn_attention_decode_workspace_bytes(int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t batch,
                                            int32_t tokens_per_seq, int32_t max_len, int32_t prefix_len)
{
    if (!heads_ok(q_heads, kv_heads, head_dim) || batch < 1 || tokens_per_seq < 1 || max_len < 0 || prefix_len < 0 ||
        (int64_t)batch * tokens_per_seq * q_heads > kI32Max)
        return 0;
    const DecodeSplit d = decode_split(q_heads, kv_heads, head_dim, batch, tokens_per_seq, max_len, prefix_len);
    return split_bytes((int64_t)batch * tokens_per_seq * q_heads, d.prefix + d.own, head_dim);
}

gdn_status gdn_attention_decode(const gdn_attention_args *args, int32_t batch, int32_t tokens_per_seq, const int32_t *lens,
                                int32_t max_len, const int32_t *prefix_table, int32_t prefix_len, void *workspace,
                                size_t workspace_bytes, void *stream)
{
    gdn::AttnDecodeParams p{};
    if (batch < 0 || tokens_per_seq < 1 || max_len < 0 || prefix_len < 0)
        return GDN_ERR_SHAPE;
    if (!args)
        return GDN_ERR_NULL;
    const int64_t queries = (int64_t)batch * tokens_per_seq;
    if (queries > kI32Max || max_len > kMaxKeys || prefix_len > gdn::kMostKeys)
        return GDN_ERR_OVERFLOW;
    const gdn_status st = check_attention(args, queries, p.a);
    if (st != GDN_OK)
        return st;
    if (args->page_size == 0)
        return GDN_ERR_UNSUPPORTED;
    if (batch == 0)
        return GDN_OK;
    if (!lens || (max_len > 0 && !args->table) || (prefix_len > 0 && !prefix_table) ||
        (max_len + (int64_t)prefix_len > 0 && (!args->k || !args->v)))
        return GDN_ERR_NULL;
    const int64_t ps = args->page_size;
    if (args->table_stride < (max_len + ps - 1) / ps || (max_len + (int64_t)prefix_len > 0 && args->num_pages < 1))
        return GDN_ERR_SHAPE;
    if (!aligned(lens, 4) || !aligned(prefix_table, 4))
        return GDN_ERR_ALIGN;
    const DecodeSplit d = decode_split(p.a.Hq, p.a.Hkv, p.a.D, batch, tokens_per_seq, max_len, prefix_len);
    if (gdn::attn_decode_blocks(p.a.Hq, p.a.Hkv, p.a.D, batch, tokens_per_seq) * d.own >= kMaxBlocks ||
        gdn::attn_prefill_blocks(p.a.Hq, p.a.Hkv, 1, queries, false) * std::max(d.prefix, 1) >= kMaxBlocks)
        return GDN_ERR_OVERFLOW;
    const int64_t rows = queries * p.a.Hq;
    const int slots = d.prefix + d.own;
    if (slots > 1 && gdn::attn_join_blocks(p.a.D, slots, rows) >= kMaxBlocks)
        return GDN_ERR_OVERFLOW;
    const size_t need = split_bytes(rows, slots, p.a.D);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return GDN_ERR_WORKSPACE;
    if (!aligned(workspace, 256))
        return GDN_ERR_ALIGN;
    carve(p.a, rows, slots, workspace);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = hipSuccess;
    if (prefix_len > 0) {
        // every query of the batch against the prefix, as one block of rows
        gdn::AttnPrefillParams f{};
        f.a = p.a;
        f.a.kv.table = prefix_table;
        f.N = 1;
        f.T = f.total = (int)queries;
        f.max_keys = prefix_len;
        f.splits = d.prefix;
        f.split_tiles = d.prefix_tiles;
        e = gdn::launch_attn_prefill(f, s);
    }
    p.B = batch;
    p.T = tokens_per_seq;
    p.lens = lens;
    p.max_len = max_len;
    p.splits = d.own;
    p.split_keys = d.own_keys;
    p.first_slot = d.prefix;
    if (e == hipSuccess)
        e = gdn::launch_attn_decode(p, s);
    if (e == hipSuccess && p.a.slots > 0)
        e = gdn::launch_attn_join(p.a, rows, s);
    return launch_status(e);
}

gdn_status gdn_pages_free(const gdn_page_args *args, int32_t n, const int32_t *rows, const int32_t *keep, void *stream)
{
    gdn::PageParams p{};
    gdn_status st = check_requests(n);
    if (st == GDN_OK)
        st = check_pages(args, false, p);
    if (st != GDN_OK || n == 0)
        return st;
    if (!rows)
        return GDN_ERR_NULL;
    if (!aligned(rows, 4) || !aligned(keep, 4))
        return GDN_ERR_ALIGN;
    p.n = n;
    p.row = rows;
    p.len = keep;
    return launch_status(gdn::launch_pages_free(p, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_pages_reserve(const gdn_page_args *args, int32_t n, const int32_t *rows, const int32_t *lens, int32_t *status,
                             void *stream)
{
    gdn::PageParams p{};
    gdn_status st = check_requests(n);
    if (st == GDN_OK)
        st = check_pages(args, false, p);
    if (st != GDN_OK)
        return st;
    if (args->page_size < 1)
        return GDN_ERR_SHAPE;
    if (n == 0)
        return GDN_OK;
    if (!rows || !lens || !status)
        return GDN_ERR_NULL;
    if (!aligned(rows, 4) || !aligned(lens, 4) || !aligned(status, 4))
        return GDN_ERR_ALIGN;
    p.n = n;
    p.row = rows;
    p.len = lens;
    p.status = status;
    return launch_status(gdn::launch_pages_reserve(p, static_cast<hipStream_t>(stream)));
}

size_t gdn_pages_workspace_bytes(int32_t num_pages)
{
    return num_pages < 0 ? 0 : gdn::pages_workspace_bytes(num_pages);
}

gdn_status gdn_pages_fork(const gdn_page_args *args, int32_t n, const int32_t *src, const int32_t *dst, const int32_t *lens,
                          int32_t *status, void *workspace, size_t workspace_bytes, void *stream)
{
    gdn::PageParams p{};
    gdn_status st = check_requests(n);
    if (st == GDN_OK)
        st = check_pages(args, true, p);
    if (st != GDN_OK)
        return st;
    if (args->page_size < 1)
        return GDN_ERR_SHAPE;
    if (n == 0)
        return GDN_OK;
    if (!src || !dst || !lens || !status)
        return GDN_ERR_NULL;
    if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(lens, 4) || !aligned(status, 4))
        return GDN_ERR_ALIGN;
    st = check_page_workspace(args, workspace, workspace_bytes);
    if (st != GDN_OK)
        return st;
    p.n = n;
    p.row = dst;
    p.src = src;
    p.len = lens;
    p.status = status;
    p.workspace = static_cast<int32_t *>(workspace);
    return launch_status(gdn::launch_pages_fork(p, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_pages_compact(const gdn_page_args *args, int32_t *page_map, int32_t *used, void *workspace, size_t workspace_bytes,
                             void *stream)
{
    gdn::PageParams p{};
    gdn_status st = check_pages(args, true, p);
    if (st != GDN_OK)
        return st;
    if (!used || (args->num_pages > 0 && !page_map))
        return GDN_ERR_NULL;
    if (!aligned(page_map, 4) || !aligned(used, 4))
        return GDN_ERR_ALIGN;
    st = check_page_workspace(args, workspace, workspace_bytes);
    if (st != GDN_OK)
        return st;
    p.page_map = page_map;
    p.used = used;
    p.workspace = static_cast<int32_t *>(workspace);
    return launch_status(gdn::launch_pages_compact(p, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
