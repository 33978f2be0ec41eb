// api_block.cu - the extern "C" entry points of the decoder-block operators
// (declared in include/w4.h): argument checks on the host, then one launch.
#include "w4_internal.h"

#include <algorithm>
#include <cmath>

namespace w4 {
namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Checks of the cache that every call shares, on a copy in which the strides
// of dimensions of extent 1 (never used) are replaced by valid ones.
int check_kv(const w4_paged_kv* in, w4_paged_kv* kv) {
    if (!in || !in->k || !in->v || !in->table || !in->kv_len) return W4_ERR_NULL_PTR;
    *kv = *in;
    if (kv->pages == 1) kv->k_page_stride = kv->v_page_stride = 8;
    if (kv->heads == 1) kv->k_head_stride = kv->v_head_stride = 8;
    if (kv->batch == 1) kv->table_stride = 0;
    if (kv->pages < 1 || kv->max_pages < 1 || kv->heads < 1 || kv->batch < 0 || kv->head_dim < 1 ||
        kv->table_stride < 0)
        return W4_ERR_INVALID_ARG;
    const int ps = kv->page_size;
    if (ps < 16 || ps > 4096 || (ps & (ps - 1))) return W4_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(kv->k, 16) || !aligned(kv->v, 16) || !aligned(kv->table, 4) || !aligned(kv->kv_len, 4))
        return W4_ERR_MISALIGNED;
    for (int64_t s : {kv->k_page_stride, kv->k_head_stride, kv->k_slot_stride, kv->v_page_stride,
                      kv->v_head_stride, kv->v_slot_stride}) {
        if (s < 1) return W4_ERR_INVALID_ARG;
        if (s % 8) return W4_ERR_MISALIGNED;
    }
    return W4_OK;
}

// The part of the attention calls' checks that does not depend on the form.  As for
// the cache, strides of extent 1 (of `tokens` and q_heads) are replaced by valid ones.
int check_attn(const w4_paged_kv* in, const uint16_t* q, long long q_tok, long long q_head,
               uint16_t* out, float* lse, int tokens, int q_heads, int max_len, float scale, int window,
               int sinks, AttnArgs* a) {
    w4_paged_kv* kv = &a->kv;
    const int rc = check_kv(in, kv);
    if (rc) return rc;
    if (!q || !out) return W4_ERR_NULL_PTR;
    if (kv->head_dim != 64 && kv->head_dim != 128) return W4_ERR_UNSUPPORTED_SHAPE;
    if (tokens == 1) q_tok = 8;
    if (q_heads == 1) q_head = 8;
    if (q_heads < 1 || q_heads % kv->heads || max_len < 0 || window < 0 || sinks < 0 || q_tok < 0 || q_head < 0 ||
        !(scale > 0.f) || !std::isfinite(scale))
        return W4_ERR_INVALID_ARG;
    // positions, windows and their differences stay inside 32 bits
    if (max_len > (1 << 30)) return W4_ERR_UNSUPPORTED_SHAPE;
    window = std::min(window, 1 << 30);
    if (q_heads / kv->heads > 128) return W4_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(q, 16) || !aligned(out, 16) || q_tok % 8 || q_head % 8 || !aligned(lse, 4))
        return W4_ERR_MISALIGNED;
    a->q = q; a->q_tok = q_tok; a->q_head = q_head;
    a->out = out; a->lse = lse; a->Hq = q_heads; a->max_len = max_len;
    a->scale = scale * 1.4426950408889634f; a->window = window; a->sinks = sinks;
    return W4_OK;
}

int attn_workspace(AttnArgs* a, size_t need, void* ws, size_t ws_bytes) {
    if (!ws || ws_bytes < kCounterBytes + need) return W4_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return W4_ERR_MISALIGNED;
    a->tickets = static_cast<int*>(ws);
    a->partial = reinterpret_cast<float*>(static_cast<char*>(ws) + kCounterBytes);
    a->err = device_error_flag();
    return a->err ? W4_OK : W4_ERR_CUDA;
}

// The scratch of w4_attn_shared, from its first 32-byte boundary on; returns its bytes.
size_t shared_scratch(AttnShared* s, void* base, int batch, int q_heads, int heads, int head_dim, int sms) {
    char* p = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(base) + 31) & ~(uintptr_t)31);
    char* const p0 = p;
    auto take = [&](size_t bytes) {
        char* at = p;
        p += (bytes + 31) & ~(size_t)31;
        return at;
    };
    const size_t rows = (size_t)batch * q_heads, slots = (size_t)2 * sms * kSharedRows;
    s->share = reinterpret_cast<int*>(take(sizeof(int)));
    s->info = reinterpret_cast<int4*>(take(batch * sizeof(int4)));
    s->row_ml = reinterpret_cast<float*>(take(rows * 2 * sizeof(float)));
    s->slot_ml = reinterpret_cast<float*>(take(slots * 2 * sizeof(float)));
    s->row_o = reinterpret_cast<float*>(take(rows * head_dim * sizeof(float)));
    s->slot_o = reinterpret_cast<float*>(take(slots * head_dim * sizeof(float)));
    const size_t own = shared_own_slots(q_heads, heads, head_dim, sms);
    s->own_share = reinterpret_cast<int*>(take(sizeof(int)));
    s->own_info = reinterpret_cast<int2*>(take(batch * sizeof(int2)));
    s->own_row_ml = reinterpret_cast<float*>(take(rows * 2 * sizeof(float)));
    s->own_slot_ml = reinterpret_cast<float*>(take(own * 2 * sizeof(float)));
    s->own_row_o = reinterpret_cast<float*>(take(rows * head_dim * sizeof(float)));
    s->own_slot_o = reinterpret_cast<float*>(take(own * head_dim * sizeof(float)));
    return (size_t)(p - p0) + 32;
}

}  // namespace
}  // namespace w4

using namespace w4;

extern "C" {

int w4_block_norm(const uint16_t* y, const uint16_t* r, const uint16_t* w_post, const uint16_t* gate,
                  const uint16_t* w_pre, uint16_t* r_out, uint16_t* x_out, int M, int K, int gate_rows,
                  float res_scale, float eps, float w_offset, void* stream) {
    if (!r || (y && !r_out) || (x_out && !w_pre) || (!y && !x_out)) return W4_ERR_NULL_PTR;
    if (!y && (w_post || gate || r_out)) return W4_ERR_INVALID_ARG;
    if (M < 0 || K < 1 || !(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(w_offset) ||
        !std::isfinite(res_scale))
        return W4_ERR_INVALID_ARG;
    if ((gate != nullptr) != (gate_rows != 0) || gate_rows < 0 || (gate && M % gate_rows)) return W4_ERR_INVALID_ARG;
    if (K > W4_BLOCK_NORM_MAX_K) return W4_ERR_UNSUPPORTED_SHAPE;
    for (const void* p : {(const void*)y, (const void*)r, (const void*)w_post, (const void*)gate, (const void*)w_pre,
                          (const void*)r_out, (const void*)x_out})
        if (!aligned(p, 2)) return W4_ERR_MISALIGNED;
    if (M == 0) return W4_OK;
    NormArgs a{};
    a.y = y; a.r = r; a.w_post = w_post; a.gate = gate; a.w_pre = w_pre;
    a.r_out = r_out; a.x_out = x_out;
    a.M = M; a.K = K; a.gate_div = gate ? M / gate_rows : 1;
    a.res_scale = res_scale; a.eps = eps; a.w_off = w_offset;
    return launch_block_norm(a, static_cast<cudaStream_t>(stream));
}

int w4_rope_freqs(int rot_dim, double base, int kind, double factor, double orig_len, double beta_fast,
                  double beta_slow, float* inv_freq, float* mscale) {
    if (!inv_freq || !mscale) return W4_ERR_NULL_PTR;
    if (rot_dim < 2 || rot_dim % 2 || !(base > 1.0) || !std::isfinite(base) || kind < W4_ROPE_PLAIN ||
        kind > W4_ROPE_YARN)
        return W4_ERR_INVALID_ARG;
    if (kind != W4_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return W4_ERR_INVALID_ARG;
    if (kind == W4_ROPE_YARN &&
        (!(orig_len >= 1.0) || !std::isfinite(orig_len) || !(beta_slow > 0.0) || !(beta_fast > beta_slow) ||
         !std::isfinite(beta_fast)))
        return W4_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925286766559;
    const int n = rot_dim / 2;
    double b = base;
    if (kind == W4_ROPE_NTK) {
        if (rot_dim < 4) return W4_ERR_INVALID_ARG;          // the exponent rot_dim / (rot_dim - 2)
        b = base * std::pow(factor, (double)rot_dim / (rot_dim - 2));
    }
    // the pair index at which a frequency turns `t` times over orig_len
    auto pair_of = [&](double t) { return rot_dim * std::log(orig_len / (t * two_pi)) / (2.0 * std::log(base)); };
    double lo = 0.0, hi = 0.0;
    if (kind == W4_ROPE_YARN) {
        lo = std::max(std::floor(pair_of(beta_fast)), 0.0);
        hi = std::min(std::ceil(pair_of(beta_slow)), (double)rot_dim - 1);
        if (hi <= lo) hi = lo + 0.001;                       // an empty ramp becomes a step
    }
    for (int i = 0; i < n; ++i) {
        double f = std::pow(b, -2.0 * i / rot_dim);
        if (kind == W4_ROPE_LINEAR) f /= factor;
        if (kind == W4_ROPE_YARN) {
            const double ramp = std::min(std::max((i - lo) / (hi - lo), 0.0), 1.0);   // 0: kept, 1: divided
            f = f * (1.0 - ramp) + f / factor * ramp;
        }
        inv_freq[i] = (float)f;
    }
    *mscale = kind == W4_ROPE_YARN && factor > 1.0 ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
    return W4_OK;
}

int w4_rope_append(const w4_paged_kv* kv, const uint16_t* q, long long q_token_stride, long long q_head_stride,
                   const uint16_t* k, long long k_token_stride, long long k_head_stride, const uint16_t* v,
                   long long v_token_stride, long long v_head_stride, const int32_t* goff, const int32_t* pos,
                   const float* inv_freq, float mscale, int rot_dim, int interleaved, uint16_t* q_out, int T,
                   int q_heads, void* stream) {
    RopeArgs a{};
    const int rc = check_kv(kv, &a.kv);
    if (rc) return rc;
    if (!q || !k || !v || !q_out || (rot_dim > 0 && !inv_freq)) return W4_ERR_NULL_PTR;
    if (T < 0 || q_heads < 1 || rot_dim < 0 || rot_dim % 2 || rot_dim > kv->head_dim || !std::isfinite(mscale))
        return W4_ERR_INVALID_ARG;
    for (long long s : {q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride, v_head_stride})
        if (s < 0) return W4_ERR_INVALID_ARG;
    if (kv->head_dim % 8 || kv->head_dim > 256) return W4_ERR_UNSUPPORTED_SHAPE;
    if (!goff && T != kv->batch) return W4_ERR_INVALID_ARG;
    for (const void* p : {(const void*)q, (const void*)k, (const void*)v, (const void*)q_out})
        if (!aligned(p, 2)) return W4_ERR_MISALIGNED;
    if (!aligned(goff, 4) || !aligned(pos, 4) || !aligned(inv_freq, 4)) return W4_ERR_MISALIGNED;
    if (T == 0 || kv->batch == 0) return W4_OK;
    a.q = q; a.k = k; a.v = v;
    a.q_tok = q_token_stride; a.q_head = q_head_stride; a.k_tok = k_token_stride; a.k_head = k_head_stride;
    a.v_tok = v_token_stride; a.v_head = v_head_stride;
    a.goff = goff; a.pos = pos; a.inv_freq = inv_freq; a.mscale = mscale; a.rot = rot_dim;
    a.inter = interleaved ? 1 : 0;
    a.q_out = q_out; a.T = T; a.Hq = q_heads;
    a.err = device_error_flag();
    if (!a.err) return W4_ERR_CUDA;
    return launch_rope_append(a, static_cast<cudaStream_t>(stream));
}

size_t w4_attn_decode_workspace_bytes(int q_heads, int heads, int head_dim) {
    if (q_heads < 1 || heads < 1 || q_heads % heads || head_dim < 1) return 0;
    const int sms = current_sm_count();
    return sms < 1 ? 0 : kCounterBytes + attn_decode_ws_bytes(q_heads, heads, head_dim, sms);
}

int w4_attn_decode(const w4_paged_kv* kv, const uint16_t* q, long long q_token_stride, long long q_head_stride,
                   uint16_t* out, float* lse, int q_heads, int max_len, float scale, int window, int sinks,
                   void* workspace, size_t workspace_bytes, void* stream) {
    AttnArgs a{};
    int rc = check_attn(kv, q, q_token_stride, q_head_stride, out, lse, kv ? kv->batch : 0, q_heads, max_len, scale,
                        window, sinks, &a);
    if (rc) return rc;
    if (kv->batch == 0) return W4_OK;
    // the list of units is counted in 32 bits
    const long long cap = std::min((long long)a.kv.max_pages * a.kv.page_size, (long long)max_len);
    if ((cap / 64 + 8) * q_heads * kv->batch > (1LL << 30)) return W4_ERR_UNSUPPORTED_SHAPE;
    const int sms = current_sm_count();
    rc = attn_workspace(&a, attn_decode_ws_bytes(q_heads, kv->heads, kv->head_dim, sms), workspace,
                        workspace_bytes);
    if (rc) return rc;
    a.T = kv->batch;
    a.max_q = 1;
    return launch_attn_decode(a, sms, static_cast<cudaStream_t>(stream));
}

int w4_attn_prefill(const w4_paged_kv* kv, const uint16_t* q, long long q_token_stride, long long q_head_stride,
                    const int32_t* goff, uint16_t* out, float* lse, int T, int q_heads, int max_q, int max_len,
                    float scale, int window, int sinks, void* stream) {
    AttnArgs a{};
    const int rc = check_attn(kv, q, q_token_stride, q_head_stride, out, lse, T, q_heads, max_len, scale, window, sinks,
                              &a);
    if (rc) return rc;
    if (!goff) return W4_ERR_NULL_PTR;
    if (T < 0 || max_q < 0) return W4_ERR_INVALID_ARG;
    if (!aligned(goff, 4)) return W4_ERR_MISALIGNED;
    if (kv->batch == 0 || T == 0 || max_q == 0) return W4_OK;
    a.err = device_error_flag();
    if (!a.err) return W4_ERR_CUDA;
    if (a.q_head == 0 || a.q_tok == 0) return W4_ERR_INVALID_ARG;
    a.goff = goff;
    a.T = T;
    a.max_q = std::min(max_q, T);
    return launch_attn_prefill(a, current_sm_count(), static_cast<cudaStream_t>(stream));
}

size_t w4_attn_shared_scratch_bytes(int batch, int q_heads, int heads, int head_dim) {
    if (batch < 0 || q_heads < 1 || heads < 1 || q_heads % heads || head_dim < 1) return 0;
    const int sms = current_sm_count();
    AttnShared sh;
    return sms < 1 ? 0 : shared_scratch(&sh, nullptr, batch, q_heads, heads, head_dim, sms);
}

int w4_attn_shared(const w4_paged_kv* kv, const uint16_t* q, long long q_token_stride, long long q_head_stride,
                   const int32_t* group, const int32_t* shared, int groups, uint16_t* out, float* lse, int q_heads,
                   int max_len, float scale, void* scratch, size_t scratch_bytes, void* stream) {
    SharedArgs a{};
    int rc = check_attn(kv, q, q_token_stride, q_head_stride, out, lse, kv ? kv->batch : 0, q_heads, max_len, scale, 0,
                        0, &a);
    if (rc) return rc;
    if (!group || !shared) return W4_ERR_NULL_PTR;
    if (groups < 1) return W4_ERR_INVALID_ARG;
    if (!aligned(group, 4) || !aligned(shared, 4)) return W4_ERR_MISALIGNED;
    if (kv->batch == 0) return W4_OK;
    if (a.q_head == 0 || a.q_tok == 0) return W4_ERR_INVALID_ARG;
    // the lists of units (blocks of 16 keys of an item of up to 8 or 16 heads; half steps of 128 are fewer) are
    // counted in 32 bits
    const int g = q_heads / a.kv.heads, items = a.kv.heads * (g <= 8 ? 1 : (g + 15) / 16);
    const long long cap = std::min((long long)a.kv.max_pages * a.kv.page_size, (long long)max_len);
    if ((cap / 16 + 8) * items > (1LL << 30) / kv->batch) return W4_ERR_UNSUPPORTED_SHAPE;
    if (!scratch) return W4_ERR_WORKSPACE;
    if (!aligned(scratch, 16)) return W4_ERR_MISALIGNED;
    const int sms = current_sm_count();
    if (scratch_bytes < shared_scratch(&a.sh, scratch, kv->batch, q_heads, kv->heads, kv->head_dim, sms)) return W4_ERR_WORKSPACE;
    a.err = device_error_flag();
    if (!a.err) return W4_ERR_CUDA;
    a.sh.group = group; a.sh.shared = shared; a.sh.groups = groups;
    a.T = kv->batch;
    a.max_q = 1;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    rc = launch_attn_shared_own(a, sms, s);
    if (rc == W4_OK) rc = launch_attn_shared_prefix(a, sms, s);
    return rc ? rc : launch_attn_shared_join(a, sms, s);
}

}  // extern "C"
