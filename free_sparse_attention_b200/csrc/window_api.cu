// C ABI of the query/key norm with 3D RoPE and of window attention with sinks: argument
// checks, workspace sizes and launches (declared in include/scope.h).
#include "qk_norm.cuh"
#include "window.cuh"

#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <atomic>
#include <cmath>

using namespace scope;

namespace {

constexpr size_t kAlign = 256;
constexpr size_t kHeader = 512;      // status word, scheduler counter
constexpr int kPlanSms = 148;        // the split plan is a function of the shape alone
constexpr int kMaxSplits = 64;

struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};

bool ok_ptr(const void *p)
{
    return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

bool ok_opt(const void *p)
{
    return !p || ok_ptr(p);
}

size_t align_up(size_t x)
{
    return (x + kAlign - 1) / kAlign * kAlign;
}

scope_status cuda_status(cudaError_t e)
{
    return e == cudaSuccess ? SCOPE_OK : SCOPE_ERR_CUDA;
}

// SMs of the current device (a property that never changes: asked once per device).
scope_status device_sms(int &sms)
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SCOPE_ERR_CUDA;
    std::atomic<int> *slot = dev >= 0 && dev < 64 ? &known[dev] : nullptr;
    if (slot && (sms = slot->load(std::memory_order_relaxed)) > 0) return SCOPE_OK;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return SCOPE_ERR_CUDA;
    if (slot) slot->store(sms, std::memory_order_relaxed);
    return SCOPE_OK;
}

// A layout (all zero: dense [B, heads, N, d]) resolved and checked: every stride of a
// dimension longer than one a positive multiple of 16 bytes, no two elements in one place.
bool layout(const scope_strides &in, long long B, long long heads, long long N, int d, int es, WinLayout &out)
{
    if (in.batch == 0 && in.head == 0 && in.token == 0) {
        out = {heads * N * d, N * d, d};
        return true;
    }
    struct Dim {
        long long stride, size;
    } dims[3] = {{in.batch, B}, {in.head, heads}, {in.token, N}};
    Dim used[3];
    int n = 0;
    for (const Dim &x : dims) {
        if (x.size == 1) continue;
        if (x.stride < d || x.stride > (1ll << 36) || (x.stride * es) % 16) return false;
        used[n++] = x;
    }
    std::sort(used, used + n, [](const Dim &x, const Dim &y) { return x.stride < y.stride; });
    long long extent = d;
    for (int k = 0; k < n; ++k) {
        if (used[k].stride < extent || used[k].size > (1ll << 40) / used[k].stride) return false;
        extent = used[k].stride * used[k].size;
    }
    // a dimension of length one is never stepped over
    out = {B == 1 ? extent : in.batch, heads == 1 ? extent : in.head, N == 1 ? extent : in.token};
    return true;
}

// ---------------------------------------------------------------------- norm + RoPE
scope_status validate(const scope_qk_norm_params *p)
{
    if (!p) return SCOPE_ERR_INVALID_ARGUMENT;
    if (p->B < 1 || p->H < 1 || p->Hkv < 1 || p->N < 1 || p->Hg < 1 || p->Wg < 1) return SCOPE_ERR_INVALID_ARGUMENT;
    if (p->d_t < 0 || p->d_h < 0 || p->d_w < 0 || p->d_t > p->d || p->d_h > p->d || p->d_w > p->d ||
        p->d_t + p->d_h + p->d_w != p->d || p->d_t % 2 || p->d_h % 2 || p->d_w % 2)
        return SCOPE_ERR_INVALID_ARGUMENT;
    if (p->d != 64 && p->d != 128) return SCOPE_ERR_UNSUPPORTED;
    if (p->dtype != SCOPE_F32 && p->dtype != SCOPE_BF16) return SCOPE_ERR_INVALID_ARGUMENT;
    if (!(p->eps >= 0.0 && p->eps <= 1.0) || !(p->base > 0.0 && std::isfinite(p->base))) return SCOPE_ERR_INVALID_ARGUMENT;
    if (p->first < 0) return SCOPE_ERR_INVALID_ARGUMENT;
    if (p->N > (1 << 24) || p->first > (1 << 30) || (long long)p->Hg * p->Wg > (1ll << 30) ||
        (long long)p->B * std::max(p->H, p->Hkv) > (1ll << 20) ||
        (long long)p->B * std::max(p->H, p->Hkv) * p->N >= (1ll << 31))
        return SCOPE_ERR_UNSUPPORTED;
    return SCOPE_OK;
}

// Turns per position of an axis of n pairs: r^i / 2 pi with r = base^(-1 / n), into f[k ..]; returns
// the end.  r's error comes back i times in r^i, so r is corrected by one Newton step of r^n = 1 / base
// and all powers are taken in long double (64 bits of mantissa): a frequency is rounded to binary64 once.
// (A long double pow for each axis takes 1.3 us of a call, this 0.15.)
int axis_frequencies(double base, int n, double *f, int k)
{
    if (n == 0) return k;
    const double r0 = std::pow(base, -1.0 / n);
    long double power = 1.0L, square = r0;
    for (int e = n; e; e >>= 1) {
        if (e & 1) power *= square;
        square *= square;
    }
    const long double r = r0 * (1.0L - (base * power - 1.0L) / n), rr = r * r;
    long double even = 0.159154943091895335768883763372514362L, odd = even * r;   // two chains side by side
    for (int i = 0; i < n; i += 2) {
        f[k++] = (double)even;
        if (i + 1 < n) f[k++] = (double)odd;
        even *= rr;
        odd *= rr;
    }
    return k;
}

scope_status norm_args(const scope_qk_norm_params &p, const int32_t *first, NormArgs &a)
{
    a.B = p.B;
    a.H = p.H;
    a.Hkv = p.Hkv;
    a.N = p.N;
    a.d = p.d;
    a.dt = p.d_t;
    a.dh = p.d_h;
    a.Hg = p.Hg;
    a.Wg = p.Wg;
    a.is_bf16 = p.dtype == SCOPE_BF16;
    a.first = first;
    a.first0 = p.first;
    a.eps = (float)p.eps;
    int k = 0;
    for (int w : {p.d_t, p.d_h, p.d_w}) k = axis_frequencies(p.base, w / 2, a.freq, k);
    return SCOPE_OK;
}

constexpr size_t norm_ws(int d)
{
    return kAlign + sizeof(float) * 2 * kNormMaxBlocks * (size_t)d;
}

// ---------------------------------------------------------------------- window attention
scope_status validate(const scope_window_params *p)
{
    if (!p) return SCOPE_ERR_INVALID_ARGUMENT;
    if (p->B < 1 || p->H < 1 || p->Hkv < 1 || p->Nq < 1 || p->Nk < 1 || p->frame < 1) return SCOPE_ERR_INVALID_ARGUMENT;
    if (p->H % p->Hkv) return SCOPE_ERR_INVALID_ARGUMENT;
    if (p->left < -1 || p->right < -1 || p->sinks < 0 || p->q_first < 0) return SCOPE_ERR_INVALID_ARGUMENT;
    if (p->dtype != SCOPE_F32 && p->dtype != SCOPE_BF16) return SCOPE_ERR_INVALID_ARGUMENT;
    if (p->d != 64 && p->d != 128) return SCOPE_ERR_UNSUPPORTED;
    if (p->Nq > (1 << 24) || p->Nk > (1 << 24) || p->frame > (1 << 24) || p->left > kWinUnbounded ||
        p->right > kWinUnbounded || p->sinks > kWinUnbounded || p->q_first > (1 << 30) ||
        (long long)p->B * p->H > (1ll << 20) || (long long)p->B * p->H * p->Nq >= (1ll << 31) ||
        (long long)p->B * p->Hkv * p->Nk >= (1ll << 31))
        return SCOPE_ERR_UNSUPPORTED;
    return SCOPE_OK;
}

// How the forward pass cuts its work: query heads whose rows share a tile, and key ranges
// per row tile.  A function of the shape alone, so that the workspace and the order of every
// sum are too.
struct Plan {
    bool few;
    int pack, splits;
};

Plan plan_of(const scope_window_params &p)
{
    Plan r;
    const int G = p.H / p.Hkv;
    // few rows: as many query heads of one key head as fill 16 rows share a tile, so that the keys
    // are read once for all of them (in equal packs)
    r.few = p.Nq <= 16;
    r.pack = 1;
    for (int n = 2; r.few && n <= G && n * p.Nq <= 16; ++n)
        if (G % n == 0) r.pack = n;
    // rows of one item and keys of one of its tiles: few rows, tensor cores, or fp32; items
    // that the plan takes the device to hold at a time (fp32 at d 128: two an SM, where the kernel has
    // come to fit three; three here is not measured)
    const bool bf16 = p.dtype == SCOPE_BF16;
    const int bm = r.few ? 16 : (bf16 ? 256 : 32), bn = r.few && bf16 ? 16 : 64;
    const int slots = kPlanSms * (bf16 ? (r.few ? 2 : 1) : (p.d == 64 ? 4 : 2));
    const long long rows = (long long)r.pack * p.Nq, tiles = (rows + bm - 1) / bm;
    const long long items = (long long)p.B * (p.H / r.pack) * tiles;
    // key tiles of one item, at most
    const long long left = p.left < 0 ? kWinUnbounded : p.left, right = p.right < 0 ? kWinUnbounded : p.right;
    const long long span = std::min((long long)p.Nk, (left + right + 1 + p.sinks) * p.frame + std::min(rows, (long long)bm));
    const long long key_tiles = (span + bn - 1) / bn;
    // Shares of an item: the count that ends first, at ceil(items * shares / slots) rounds of
    // ceil(tiles / shares) tiles and a fixed cost of about four 64-key tiles (start, store, join)
    r.splits = 1;
    const long long fixed = 256 / bn;
    // few rows in bf16: a second kernel that joins costs as much again
    const int joined = r.few && bf16 ? kFewCluster : kMaxSplits;
    long long best = -1;
    for (int n = 1; n <= kMaxSplits && (n == 1 || n * (128 / bn) <= key_tiles); ++n) {
        const long long cost = ((items * n + slots - 1) / slots) * ((key_tiles + n - 1) / n + fixed) + (n > joined ? fixed : 0);
        if (best < 0 || cost < best) {
            best = cost;
            r.splits = n;
        }
    }
    return r;
}

// Shares of the key tiles in dK, dV: a share is at most half of what a mean SM has to walk, so that
// the few tiles that all queries see do not end last (a quarter in fp32, whose SMs hold several
// blocks), and no shorter than 8 column tiles.  Of the shape alone.  Measured: bf16, 3 x 4 key heads x
// 4001, groups of 4, window 1024, 4 sinks (a tile of sinks walks 252 column tiles, the mean SM 211):
// 234 us against 331 without shares; 16 heads x 2000, window 300, a step: 97 us, with shares of 16 or
// more 100.  fp32, 8 heads x 1430, frames of 143: 410 us, with at most half 455.
KeyShares shares_of(const scope_window_params &p)
{
    const long long tile = p.dtype == SCOPE_BF16 ? 128 : 32, G = p.H / p.Hkv;
    const long long left = p.left < 0 ? kWinUnbounded : p.left, right = p.right < 0 ? kWinUnbounded : p.right;
    KeyShares k{};
    k.units = p.B * p.Hkv;
    k.tiles = (int)((p.Nk + tile - 1) / tile);
    k.sink = (int)std::min((long long)k.tiles, ((long long)p.sinks * p.frame + tile - 1) / tile);
    // column tiles that one key tile walks, at most
    const long long all = (p.Nq + 63) / 64, seen = std::min(all, (std::min((left + right + 1) * p.frame, 1ll << 24) + tile + 63) / 64 + 1);
    const long long walk[2] = {G * all, G * seen};
    const long long mean = k.units * (k.sink * walk[0] + (k.tiles - k.sink) * walk[1]) / kPlanSms;
    const long long most = std::max(8ll, mean / (p.dtype == SCOPE_BF16 ? 2 : 4));
    k.of_sink = (int)((walk[0] + most - 1) / most);
    k.of_other = (int)((walk[1] + most - 1) / most);
    return k;
}

struct WinWs {
    size_t part_o, part_lse, delta, nlse, part_kv, total;
};

WinWs ws_of(const scope_window_params &p)
{
    const Plan pl = plan_of(p);
    const size_t rows = (size_t)p.B * p.H * p.Nq;
    WinWs w;
    size_t o = kHeader;
    w.part_o = o;
    if (pl.splits > 1) o = align_up(o + sizeof(float) * rows * pl.splits * p.d);
    w.part_lse = o;
    if (pl.splits > 1) o = align_up(o + sizeof(float) * rows * pl.splits);
    w.delta = kHeader;   // the backward pass has the partials' place to itself
    w.nlse = align_up(w.delta + sizeof(float) * rows);
    w.part_kv = p.dtype == SCOPE_BF16 ? align_up(w.nlse + sizeof(float) * rows) : w.nlse;
    w.total = std::max(o, w.part_kv + sizeof(float) * 2 * (p.dtype == SCOPE_BF16 ? 128 : 32) * p.d * (size_t)shares_of(p).parts());
    return w;
}

scope_status window_args(const scope_window_params &p, const scope_window_layouts *lay, const int32_t *q_first,
                         const int32_t *k_len, void *ws, bool backward, WinArgs &a)
{
    const scope_window_layouts dense{}, &L = lay ? *lay : dense;
    const int es = p.dtype == SCOPE_BF16 ? 2 : 4;
    bool ok = layout(L.q, p.B, p.H, p.Nq, p.d, es, a.lq) && layout(L.k, p.B, p.Hkv, p.Nk, p.d, es, a.lk) &&
              layout(L.v, p.B, p.Hkv, p.Nk, p.d, es, a.lv) && layout(L.o, p.B, p.H, p.Nq, p.d, es, a.lo);
    if (backward)
        ok = ok && layout(L.d_o, p.B, p.H, p.Nq, p.d, es, a.lg) && layout(L.dq, p.B, p.H, p.Nq, p.d, es, a.ldq) &&
             layout(L.dk, p.B, p.Hkv, p.Nk, p.d, es, a.ldk) && layout(L.dv, p.B, p.Hkv, p.Nk, p.d, es, a.ldv);
    if (!ok) return SCOPE_ERR_INVALID_ARGUMENT;
    const Plan pl = plan_of(p);
    const WinWs w = ws_of(p);
    char *base = static_cast<char *>(ws);
    a.q_first = q_first;
    a.k_len = k_len;
    a.first0 = p.q_first;
    a.B = p.B;
    a.H = p.H;
    a.Hkv = p.Hkv;
    a.Nq = p.Nq;
    a.Nk = p.Nk;
    a.d = p.d;
    a.is_bf16 = p.dtype == SCOPE_BF16;
    a.frame = p.frame;
    a.left = p.left < 0 ? kWinUnbounded : p.left;
    a.right = p.right < 0 ? kWinUnbounded : p.right;
    a.sinks = p.sinks;
    a.pack = pl.pack;
    a.splits = pl.splits;
    a.part_o = reinterpret_cast<float *>(base + w.part_o);
    a.part_lse = reinterpret_cast<float *>(base + w.part_lse);
    a.delta = reinterpret_cast<float *>(base + w.delta);
    a.nlse = reinterpret_cast<float *>(base + w.nlse);
    a.kv = shares_of(p);
    a.kv.part = reinterpret_cast<float *>(base + w.part_kv);
    a.scale = (float)(1.0 / std::sqrt((double)p.d));
    a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)p.d));
    a.status = reinterpret_cast<int32_t *>(base);
    a.counter = reinterpret_cast<int32_t *>(base + 256);
    a.wait_ns = kTcWaitDefaultNs;
    return device_sms(a.num_sms);
}

}  // namespace

extern "C" {

size_t scope_qk_norm_workspace_bytes(const scope_qk_norm_params *p)
{
    return validate(p) == SCOPE_OK ? norm_ws(p->d) : 0;
}

scope_status scope_qk_norm_rope3d(const scope_qk_norm_params *p, const scope_qk_norm_layouts *lay, const void *Q,
                                  const void *K, const float *w_q, const float *w_k, const int32_t *first, void *Yq,
                                  void *Yk, void *stream)
{
    NvtxRange nvtx("scope_qk_norm_rope3d");
    scope_status st = validate(p);
    if (st != SCOPE_OK) return st;
    if (!ok_ptr(Q) || !ok_ptr(Yq) || !ok_opt(K) || !ok_opt(Yk) || (!K) != (!Yk) || !ok_opt(w_q) || !ok_opt(w_k) ||
        !ok_opt(first))
        return SCOPE_ERR_INVALID_ARGUMENT;
    const scope_qk_norm_layouts dense{}, &L = lay ? *lay : dense;
    const int es = p->dtype == SCOPE_BF16 ? 2 : 4;
    NormArgs a{};
    if (!layout(L.q, p->B, p->H, p->N, p->d, es, a.q.lx) || !layout(L.yq, p->B, p->H, p->N, p->d, es, a.q.ly) ||
        !layout(L.k, p->B, p->Hkv, p->N, p->d, es, a.k.lx) || !layout(L.yk, p->B, p->Hkv, p->N, p->d, es, a.k.ly))
        return SCOPE_ERR_INVALID_ARGUMENT;
    int sms = 0;
    if ((st = norm_args(*p, first, a)) != SCOPE_OK || (st = device_sms(sms)) != SCOPE_OK) return st;
    a.q.X = Q;
    a.q.Y = Yq;
    a.q.w = w_q;
    a.k.X = K;
    a.k.Y = Yk;
    a.k.w = w_k;
    return cuda_status(qk_norm_forward(a, sms, static_cast<cudaStream_t>(stream)));
}

scope_status scope_qk_norm_rope3d_backward(const scope_qk_norm_params *p, const scope_qk_norm_layouts *lay,
                                           const void *Q, const void *K, const float *w_q, const float *w_k,
                                           const void *dYq, const void *dYk, const int32_t *first, void *dQ, void *dK,
                                           float *dw_q, float *dw_k, void *ws, size_t ws_bytes, void *stream)
{
    NvtxRange nvtx("scope_qk_norm_rope3d_backward");
    scope_status st = validate(p);
    if (st != SCOPE_OK) return st;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1))) return SCOPE_ERR_INVALID_ARGUMENT;
    if (ws_bytes < norm_ws(p->d)) return SCOPE_ERR_WORKSPACE_TOO_SMALL;
    if (!ok_ptr(Q) || !ok_ptr(dYq) || !ok_ptr(dQ) || !ok_opt(K) || !ok_opt(dYk) || !ok_opt(dK) || (!K) != (!dYk) ||
        (!K) != (!dK) || !ok_opt(w_q) || !ok_opt(w_k) || !ok_opt(dw_q) || !ok_opt(dw_k) || (!K && dw_k) || !ok_opt(first))
        return SCOPE_ERR_INVALID_ARGUMENT;
    const scope_qk_norm_layouts dense{}, &L = lay ? *lay : dense;
    const int es = p->dtype == SCOPE_BF16 ? 2 : 4;
    NormArgs a{};
    if (!layout(L.q, p->B, p->H, p->N, p->d, es, a.q.lx) || !layout(L.yq, p->B, p->H, p->N, p->d, es, a.q.lg) ||
        !layout(L.dq, p->B, p->H, p->N, p->d, es, a.q.ly) || !layout(L.k, p->B, p->Hkv, p->N, p->d, es, a.k.lx) ||
        !layout(L.yk, p->B, p->Hkv, p->N, p->d, es, a.k.lg) || !layout(L.dk, p->B, p->Hkv, p->N, p->d, es, a.k.ly))
        return SCOPE_ERR_INVALID_ARGUMENT;
    int sms = 0;
    if ((st = norm_args(*p, first, a)) != SCOPE_OK || (st = device_sms(sms)) != SCOPE_OK) return st;
    a.q.X = Q;
    a.q.G = dYq;
    a.q.Y = dQ;
    a.q.w = w_q;
    a.q.dw = dw_q;
    a.k.X = K;
    a.k.G = dYk;
    a.k.Y = dK;
    a.k.w = w_k;
    a.k.dw = dw_k;
    a.status = static_cast<int32_t *>(ws);
    a.partial = reinterpret_cast<float *>(static_cast<char *>(ws) + kAlign);
    return cuda_status(qk_norm_backward(a, sms, static_cast<cudaStream_t>(stream)));
}

size_t scope_window_workspace_bytes(const scope_window_params *p)
{
    return validate(p) == SCOPE_OK ? ws_of(*p).total : 0;
}

scope_status scope_window_attention(const scope_window_params *p, const scope_window_layouts *lay, const void *Q,
                                    const void *K, const void *V, const int32_t *q_first, const int32_t *k_len, void *O,
                                    float *lse, void *ws, size_t ws_bytes, void *stream)
{
    NvtxRange nvtx("scope_window_attention");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    scope_status st = validate(p);
    if (st != SCOPE_OK) return st;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1))) return SCOPE_ERR_INVALID_ARGUMENT;
    if (ws_bytes < ws_of(*p).total) return SCOPE_ERR_WORKSPACE_TOO_SMALL;
    if (!ok_ptr(Q) || !ok_ptr(K) || !ok_ptr(V) || !ok_ptr(O) || !ok_opt(lse) || !ok_opt(q_first) || !ok_opt(k_len))
        return SCOPE_ERR_INVALID_ARGUMENT;
    WinArgs a{};
    if ((st = window_args(*p, lay, q_first, k_len, ws, false, a)) != SCOPE_OK) return st;
    a.Q = Q;
    a.K = K;
    a.V = V;
    a.O = O;
    a.lse = lse;
    if (a.is_bf16 && plan_of(*p).few) return cuda_status(window_few_forward(a, s));   // joins its shares itself
    cudaError_t e = a.is_bf16 ? window_tc_forward(a, s) : window_simt_forward(a, s);
    if (e == cudaSuccess && a.splits > 1) e = window_join(a, s);
    return cuda_status(e);
}

scope_status scope_window_attention_backward(const scope_window_params *p, const scope_window_layouts *lay,
                                             const void *Q, const void *K, const void *V, const void *O, const void *dO,
                                             const float *lse, const int32_t *q_first, const int32_t *k_len, void *dQ,
                                             void *dK, void *dV, void *ws, size_t ws_bytes, void *stream)
{
    NvtxRange nvtx("scope_window_attention_backward");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    scope_status st = validate(p);
    if (st != SCOPE_OK) return st;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1))) return SCOPE_ERR_INVALID_ARGUMENT;
    if (ws_bytes < ws_of(*p).total) return SCOPE_ERR_WORKSPACE_TOO_SMALL;
    if (!ok_ptr(Q) || !ok_ptr(K) || !ok_ptr(V) || !ok_ptr(O) || !ok_ptr(dO) || !ok_ptr(lse) || !ok_ptr(dQ) ||
        !ok_ptr(dK) || !ok_ptr(dV) || !ok_opt(q_first) || !ok_opt(k_len))
        return SCOPE_ERR_INVALID_ARGUMENT;
    WinArgs a{};
    if ((st = window_args(*p, lay, q_first, k_len, ws, true, a)) != SCOPE_OK) return st;
    a.Q = Q;
    a.K = K;
    a.V = V;
    a.O = const_cast<void *>(O);
    a.G = dO;
    a.lse = const_cast<float *>(lse);
    a.dQ = dQ;
    a.dK = dK;
    a.dV = dV;
    return cuda_status(a.is_bf16 ? window_tc_backward(a, s) : window_simt_backward(a, s));
}

}  // extern "C"
