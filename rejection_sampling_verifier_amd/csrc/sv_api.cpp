// Host side of the specverify C ABI: argument checks, scratch management,
// kernel dispatch and optional per-kernel timing.  The operation itself is
// described in include/specverify.h.

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <limits>
#include <map>
#include <mutex>
#include <string>
#include <tuple>
#include <utility>
#include <vector>

#include "../../include/specverify.h"
#include "sv_beam.h"
#include "sv_internal.h"
#include "sv_latent.h"
#include "sv_tree.h"

namespace {

using sv::Params;

struct Scratch {
    void* ptr = nullptr;       // records and per-row state; zeroed when allocated
    size_t bytes = 0;
};

static_assert(SPECVERIFY_MAX_V == sv::kMaxV, "vocabulary limit");

struct Layout {
    size_t prec, rv, qrec, chdr, cand, cum, etab, total;
};

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Tagged records (statistics per chunk, masses per resample item) carry the
// call's tag; RvState is rewritten before it is read.  The top-p candidate headers and lists (present only
// when `topp`) are rewritten by the statistics pass of every top-p call.
Layout layout(int64_t B, int nslot, int nch, int nq, int qwords, bool topp, bool smc, bool tab) {
    Layout L;
    size_t off = 0;
    L.prec = off;
    off = align256(off + static_cast<size_t>(B) * nslot * nch * sv::kRecWords * sizeof(uint64_t));
    L.rv = off;
    off = align256(off + static_cast<size_t>(B) * nslot * sizeof(sv::RvState));
    L.qrec = off;
    off = align256(off + static_cast<size_t>(B) * nq * qwords * sizeof(uint64_t));
    const size_t chunks = topp ? static_cast<size_t>(B) * nslot * nch : 0;
    L.chdr = off;
    off = align256(off + chunks * sv::kWaves * 4 * sizeof(uint64_t));  // four tagged words per wave
    L.cand = off;
    off = align256(off + chunks * sv::kCand * sizeof(uint64_t));
    L.cum = off;
    off = align256(off + (smc ? static_cast<size_t>(B) * sizeof(double) : 0));
    L.etab = off;
    off = align256(off + (tab ? static_cast<size_t>(sv::kTabN) * sizeof(double) : 0));
    L.total = off;
    return L;
}

// Record tags: unique per call within the process, never 0.
std::atomic<uint32_t> g_tag{0};
uint32_t next_tag() {
    uint32_t t;
    do {
        t = g_tag.fetch_add(1u) + 1u;
    } while (t == 0u);
    return t;
}

std::mutex g_mu;
std::map<std::pair<int, hipStream_t>, Scratch> g_scratch;
thread_local std::string g_hip_msg;

struct EvPair {
    hipEvent_t a, b;
    int kind;
};
bool g_prof = false;
std::vector<EvPair> g_events;

int hip_fail(hipError_t e, const char* what) {
    g_hip_msg = std::string(what) + ": " + hipGetErrorString(e);
    return SV_EHIP;
}

int env_int(const char* name, int dflt) {
    const char* s = std::getenv(name);
    if (!s || !*s) return dflt;
    return std::atoi(s);
}

double env_double(const char* name, double dflt) {
    const char* s = std::getenv(name);
    if (!s || !*s) return dflt;
    return std::atof(s);
}

bool misaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

// Compute units of the current device (cached per device).
int device_cus() {
    static std::mutex mu;
    static std::map<int, int> cache;
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return 256;
    std::lock_guard<std::mutex> lk(mu);
    auto it = cache.find(dev);
    if (it != cache.end()) return it->second;
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
    cache[dev] = n;
    return n;
}

int check_logits(const sv_logits* t) {
    if (!t || !t->data) return SV_EINVAL;
    if (t->dtype != SV_F32 && t->dtype != SV_BF16) return SV_EDTYPE;
    if (t->stride_b < 0 || t->stride_p < 0) return SV_EINVAL;
    if (misaligned(t->data, t->dtype == SV_BF16 ? 2 : 4)) return SV_EALIGN;
    return SV_OK;
}

// Test-only fault injection: with SPECVERIFY_FAIL_LAUNCH set to a non-zero
// value every call fails where it would first touch the device, as a failed
// launch does (SV_EHIP and its message), so that the error path can be
// tested without a GPU.
bool fail_launch_forced() { return env_int("SPECVERIFY_FAIL_LAUNCH", 0) != 0; }

// Scratch of spec_verify_noalloc: one fixed array per device, held until the
// process ends.  Host code never uses the array's name as an address (on the
// host it is only a stand-in): each device's address comes from
// hipGetSymbolAddress, taken once per device with that device current.
constexpr size_t kNoAllocBytes = static_cast<size_t>(SPECVERIFY_NOALLOC_SCRATCH_BYTES);
static __device__ __align__(256) uint8_t scratch[kNoAllocBytes];
std::mutex g_noalloc_mu;
std::map<int, void*> g_noalloc_ptr;

int noalloc_scratch(void** out) {
    if (fail_launch_forced()) return hip_fail(hipErrorLaunchFailure, "kernel launch (forced by SPECVERIFY_FAIL_LAUNCH)");
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
    std::lock_guard<std::mutex> lk(g_noalloc_mu);
    auto it = g_noalloc_ptr.find(dev);
    if (it == g_noalloc_ptr.end()) {
        void* ptr = nullptr;
        e = hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch));
        if (e != hipSuccess || ptr == nullptr) return hip_fail(e, "hipGetSymbolAddress(scratch)");
        it = g_noalloc_ptr.emplace(dev, ptr).first;
    }
    *out = it->second;
    return SV_OK;
}

// Buffers replaced by larger ones.  A HIP graph captured from an earlier
// call may still use them, so they are freed only by spec_verify_release.
std::vector<void*> g_retired;

// Returns the scratch for (device, stream), growing it (zeroed) when needed.
// Growing allocates and synchronises the stream, which a stream being
// captured into a graph cannot do: then SV_ECAPTURE, and nothing changes.
int get_scratch(hipStream_t stream, size_t bytes, void** data) {
    if (fail_launch_forced()) return hip_fail(hipErrorLaunchFailure, "kernel launch (forced by SPECVERIFY_FAIL_LAUNCH)");
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
    std::lock_guard<std::mutex> lk(g_mu);
    Scratch& s = g_scratch[{dev, stream}];
    if (s.bytes >= bytes) {
        *data = s.ptr;
        return SV_OK;
    }
    hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
    e = hipStreamIsCapturing(stream, &cap);
    if (e != hipSuccess) return hip_fail(e, "hipStreamIsCapturing");
    if (cap != hipStreamCaptureStatusNone) return SV_ECAPTURE;
    if (s.ptr) {
        e = hipStreamSynchronize(stream);
        if (e != hipSuccess) return hip_fail(e, "hipStreamSynchronize");
    }
    void* p = nullptr;
    const size_t want = bytes + bytes / 4;
    e = hipMalloc(&p, want);
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return SV_ENOMEM;
    }
    e = hipMemsetAsync(p, 0, want, stream);
    if (e != hipSuccess) {
        (void)hipFree(p);
        return hip_fail(e, "hipMemsetAsync");
    }
    if (s.ptr) g_retired.push_back(s.ptr);
    s.ptr = p;
    s.bytes = want;
    *data = s.ptr;
    return SV_OK;
}

// What a C entry point returns: no exception passes it (a host allocation that
// fails, for a message or a map's entry).
template <typename F>
auto entry(F&& call) noexcept -> decltype(call()) {
    try {
        return call();
    } catch (...) {
        return SV_ENOMEM;
    }
}

template <typename F>
int timed_launch(int kind, hipStream_t stream, F&& launch) {
    EvPair ev{nullptr, nullptr, kind};
    if (g_prof) {
        if (hipEventCreate(&ev.a) != hipSuccess || hipEventCreate(&ev.b) != hipSuccess)
            return hip_fail(hipGetLastError(), "hipEventCreate");
    }
    if (fail_launch_forced()) return hip_fail(hipErrorLaunchFailure, "kernel launch (forced by SPECVERIFY_FAIL_LAUNCH)");
    const hipError_t e = launch(sv::LaunchEvents{ev.a, ev.b});
    if (e != hipSuccess) return hip_fail(e, "kernel launch");
    if (g_prof) {
        std::lock_guard<std::mutex> lk(g_mu);
        g_events.push_back(ev);
    }
    return SV_OK;
}

// What every entry point shares: argument checks, chunking and the kernel
// parameters (plan), then the scratch pointers (bind).  `smc`: an SMC-SD step
// (no draft lengths, no top-p, the resampling kernel's scratch).
struct Setup {
    Params p;
    int dtype = 0;
    int unroll = 0;
    bool topp = false;
    hipStream_t stream = nullptr;
    Layout lay;
    bool tab = false;
};

enum Mode { MODE_VERIFY = 0, MODE_SMC = 1, MODE_GREEDY = 2 };

int plan(const sv_logits* tl, const sv_logits* dl, const int32_t* draft_tokens, const int32_t* draft_len,
         float temperature, float top_p, uint64_t seed, int mode, void* stream_v, Setup& S) {
    const bool smc = mode == MODE_SMC, greedy = mode == MODE_GREEDY;
    int rc = check_logits(tl);
    if (rc) return rc;
    if (!greedy) {
        rc = check_logits(dl);
        if (rc) return rc;
    }
    if (!draft_tokens) return SV_EINVAL;
    if (misaligned(draft_tokens, 4) || (draft_len && misaligned(draft_len, 4))) return SV_EALIGN;
    if (!greedy && tl->dtype != dl->dtype) return SV_EDTYPE;
    const int B = tl->B, V = tl->V, K = tl->P - 1;
    if (B <= 0 || V <= 0 || K < 1 || K > SPECVERIFY_MAX_K) return SV_ESHAPE;
    if (!greedy && (dl->B != B || dl->V != V || dl->P != K)) return SV_ESHAPE;
    if (B > (1 << 22) || V > (greedy ? (1 << 24) : SPECVERIFY_MAX_V)) return SV_ESHAPE;
    if (!(temperature > 0.f) || !std::isfinite(temperature)) return SV_EINVAL;
    if (!(top_p > 0.f && top_p <= 1.f)) return SV_EINVAL;
    const double c = 1.4426950408889634074 / static_cast<double>(temperature);  // log2(e)/T
    if (!(c < static_cast<double>(FLT_MAX))) return SV_EINVAL;

    const int dtype = tl->dtype == SV_BF16 ? sv::DT_BF16 : sv::DT_F32;
    const int E = dtype == sv::DT_BF16 ? 2 : 4;
    // greedy verify reads the target rows only
    const int nslot = greedy ? K + 1 : 2 * K + 1;
    // statistics pass: chunks of at most `cv` 16-byte vectors per workgroup
    const int64_t nvec_max = (static_cast<int64_t>(V) * E + 15) / 16 + 1;
    int unroll = env_int("SPECVERIFY_STATS_UNROLL", sv::kStatsUnroll);
    if (unroll != 4) unroll = 8;
    // a statistics workgroup reads one chunk of kThreads*unroll vectors; only
    // a row's last chunk is partial
    const int cv = sv::kThreads * unroll;
    const int64_t nch64 = (nvec_max + cv - 1) / cv;
    const int nch = static_cast<int>(nch64);
    // row pass: items of runs*kRunIds ids.  Four-run items by default; one-run
    // items when the batch would otherwise give fewer than two workgroups per
    // CU; sixteen-run items when four-run items would not all be resident at
    // once (four workgroups per CU), so that every row pays the pass's latency
    // chain once instead of once per round of workgroups
    int runs = sv::kRunsMax;
    if (!greedy) {
        const int cus = device_cus();
        auto items = [&](int ru) { return static_cast<int64_t>(B) * ((V + ru * sv::kRunIds - 1) / (ru * sv::kRunIds)); };
        if (items(runs) < 2ll * cus) runs = 1;
        else if (items(runs) > 4ll * cus && items(sv::kRunsBig) < items(runs)) runs = sv::kRunsBig;
        const int forced = env_int("SPECVERIFY_ROW_RUNS", 0);
        if (forced == 1 || forced == 2 || forced == sv::kRunsMax || forced == sv::kRunsBig) runs = forced;
    }
    const int nq = greedy ? 0 : (V + runs * sv::kRunIds - 1) / (runs * sv::kRunIds);
    const int qwords = sv::qrec_words(runs);
    const int64_t per_row = static_cast<int64_t>(nslot) * nch + nq;
    if (static_cast<int64_t>(B) * per_row >= (1ll << 31)) return SV_ESHAPE;
    // the statistics kernel clears the row pass's records, a few words each
    if (static_cast<int64_t>(qwords) * nq > static_cast<int64_t>(sv::kThreads) * nslot * nch) return SV_ESHAPE;

    // greedy verify takes its argmaxes and top-k from the candidate lists
    const bool topp = top_p < 1.f || greedy;
    // the top-p row pass's exponential table (bfloat16 rows; for larger c its
    // entries 2^(u*c) would leave the float64 range)
    S.tab = dtype == sv::DT_BF16 && !greedy && !smc && top_p < 1.f && c <= sv::kTabMaxC;
    S.lay = layout(B, nslot, nch, nq, qwords, topp, smc, S.tab);

    Params& p = S.p;
    std::memset(&p, 0, sizeof(p));
    p.tgt = static_cast<const uint8_t*>(tl->data);
    p.tsb = tl->stride_b;
    p.tsp = tl->stride_p;
    if (!greedy) {
        p.dft = static_cast<const uint8_t*>(dl->data);
        p.dsb = dl->stride_b;
        p.dsp = dl->stride_p;
    }
    p.tokens = draft_tokens;
    p.dlen = draft_len;
    p.B = B;
    p.K = K;
    p.V = V;
    p.nslot = nslot;
    p.nch = nch;
    p.cv = cv;
    p.nq = nq;
    p.runs = runs;
    p.qwords = qwords;
    p.tag = next_tag();
    // c = c_hi + c_lo with c_hi <= c rounded toward zero, so c_lo > 0.
    float c_hi = static_cast<float>(c);
    if (static_cast<double>(c_hi) > c) c_hi = std::nextafter(c_hi, 0.f);
    float c_lo = static_cast<float>(c - static_cast<double>(c_hi));
    if (!(c_lo >= FLT_MIN)) c_lo = FLT_MIN;
    p.c_hi = c_hi;
    p.c_lo = c_lo;
    p.c64 = c;
    // relative error bound of keptT/keptD as the statistics (and nucleus)
    // passes compute them: float32 exponentials and float32 lane and wave
    // sums, below 1.2e-6 per normaliser (below 2e-6 per kept mass)
    // SPECVERIFY_AMB_BAND replaces it (tests: 0 sends every row to the exact
    // second round, a wide band fills the items' ambiguous groups)
    p.amb_band = env_double("SPECVERIFY_AMB_BAND", top_p < 1.f ? 4e-6 : 2.5e-6);
    p.inv_c = static_cast<float>(1.0 / c);
    p.top_p = top_p;
    p.key0 = static_cast<uint32_t>(seed & 0xFFFFFFFFull);
    p.key1 = static_cast<uint32_t>(seed >> 32);
    p.smc = smc ? 1 : 0;
    S.dtype = dtype;
    S.unroll = unroll;
    S.topp = topp;
    S.stream = static_cast<hipStream_t>(stream_v);
    return SV_OK;
}

void bind(Setup& S, uint8_t* base) {
    Params& p = S.p;
    const Layout& lay = S.lay;
    p.prec = reinterpret_cast<uint64_t*>(base + lay.prec);
    p.rv = reinterpret_cast<sv::RvState*>(base + lay.rv);
    p.qrec = reinterpret_cast<uint64_t*>(base + lay.qrec);
    p.chdr = S.topp ? reinterpret_cast<uint64_t*>(base + lay.chdr) : nullptr;
    p.cand = S.topp ? reinterpret_cast<uint64_t*>(base + lay.cand) : nullptr;
    p.smc_cum = p.smc ? reinterpret_cast<double*>(base + lay.cum) : nullptr;
    p.etab = S.tab ? reinterpret_cast<double*>(base + lay.etab) : nullptr;
}

// plan + scratch + bind for a single pass.
int prepare(const sv_logits* tl, const sv_logits* dl, const int32_t* draft_tokens, const int32_t* draft_len,
            float temperature, float top_p, uint64_t seed, int mode, void* stream_v, Setup& S) {
    int rc = plan(tl, dl, draft_tokens, draft_len, temperature, top_p, seed, mode, stream_v, S);
    if (rc) return rc;
    void* scratch = nullptr;
    rc = get_scratch(S.stream, S.lay.total, &scratch);
    if (rc) return rc;
    bind(S, static_cast<uint8_t*>(scratch));
    return SV_OK;
}

// The verify step's kernels for one planned and bound pass.
int launch_verify(Setup& S) {
    Params& p = S.p;
    const hipStream_t stream = S.stream;
    int rc = timed_launch(sv::KK_STATS, stream, [&](const sv::LaunchEvents& ev) {
        return sv::launch_stats(p, S.dtype, S.unroll, S.topp, stream, ev);
    });
    if (rc) return rc;
    if (S.topp) {
        rc = timed_launch(sv::KK_TOPP, stream,
                          [&](const sv::LaunchEvents& ev) { return sv::launch_topp(p, S.dtype, stream, ev); });
        if (rc) return rc;
    }
    return timed_launch(sv::KK_RESAMPLE, stream,
                        [&](const sv::LaunchEvents& ev) { return sv::launch_rows(p, S.dtype, S.topp, stream, ev); });
}

int verify_impl(const sv_logits* tl, const sv_logits* dl, const int32_t* draft_tokens, const int32_t* draft_len,
                float temperature, float top_p, uint64_t seed, int32_t* out_tokens, int32_t* out_n,
                double* probe_pos, double* probe_row, void* stream_v) {
    if (!out_tokens || !out_n) return SV_EINVAL;
    if (misaligned(out_tokens, 4) || misaligned(out_n, 4)) return SV_EALIGN;
    Setup S;
    int rc = prepare(tl, dl, draft_tokens, draft_len, temperature, top_p, seed, MODE_VERIFY, stream_v, S);
    if (rc) return rc;
    S.p.out_tokens = out_tokens;
    S.p.out_n = out_n;
    S.p.probe_pos = probe_pos;
    S.p.probe_row = probe_row;
    return launch_verify(S);
}

// spec_verify on the fixed per-device scratch: the same kernels, no
// allocation; calls needing more than the array holds are refused.
int verify_noalloc_impl(const sv_logits* tl, const sv_logits* dl, const int32_t* draft_tokens,
                        const int32_t* draft_len, float temperature, float top_p, uint64_t seed, int32_t* out_tokens,
                        int32_t* out_n, void* stream_v) {
    if (!out_tokens || !out_n) return SV_EINVAL;
    if (misaligned(out_tokens, 4) || misaligned(out_n, 4)) return SV_EALIGN;
    Setup S;
    int rc = plan(tl, dl, draft_tokens, draft_len, temperature, top_p, seed, MODE_VERIFY, stream_v, S);
    if (rc) return rc;
    if (S.lay.total > kNoAllocBytes) return SV_ETOOBIG;
    void* base = nullptr;
    rc = noalloc_scratch(&base);
    if (rc) return rc;
    bind(S, static_cast<uint8_t*>(base));
    S.p.out_tokens = out_tokens;
    S.p.out_n = out_n;
    return launch_verify(S);
}

// Two-stage verify: stage 1 verifies the drafts against the intermediate
// layer, stage 2 the n1 + 1 tokens it emitted against the final layer (the
// intermediate layer as their proposal, Philox stream 1).  One scratch
// allocation holds both passes' regions and stage 1's outputs.
int hispec_impl(const sv_logits* fl, const sv_logits* il, const sv_logits* dl, const int32_t* draft_tokens,
                const int32_t* draft_len, float temperature, float top_p, uint64_t seed, int32_t* out_tokens,
                int32_t* out_n, int32_t* out_n_stage1, void* stream_v) {
    if (!out_tokens || !out_n) return SV_EINVAL;
    if (misaligned(out_tokens, 4) || misaligned(out_n, 4) || (out_n_stage1 && misaligned(out_n_stage1, 4)))
        return SV_EALIGN;
    if (!fl || !il) return SV_EINVAL;
    if (fl->B != il->B || fl->V != il->V || fl->P != il->P + 1) return SV_ESHAPE;
    Setup S1, S2;
    int rc = plan(il, dl, draft_tokens, draft_len, temperature, top_p, seed, MODE_VERIFY, stream_v, S1);
    if (rc) return rc;
    // stage 2's drafts are device scratch bound below; the caller's ids stand
    // in for the host checks
    rc = plan(fl, il, draft_tokens, nullptr, temperature, top_p, seed, MODE_VERIFY, stream_v, S2);
    if (rc) return rc;
    const int B = S1.p.B, K1 = S1.p.K + 1;
    const size_t tok_bytes = align256(static_cast<size_t>(B) * K1 * sizeof(int32_t));
    const size_t vec_bytes = align256(static_cast<size_t>(B) * sizeof(int32_t));
    const size_t total = S1.lay.total + S2.lay.total + tok_bytes + 2 * vec_bytes;
    void* scratch = nullptr;
    rc = get_scratch(S1.stream, total, &scratch);
    if (rc) return rc;
    uint8_t* base = static_cast<uint8_t*>(scratch);
    bind(S1, base);
    bind(S2, base + S1.lay.total);
    uint8_t* extra = base + S1.lay.total + S2.lay.total;
    int32_t* tok1 = reinterpret_cast<int32_t*>(extra);
    int32_t* n1 = reinterpret_cast<int32_t*>(extra + tok_bytes);
    int32_t* len2 = reinterpret_cast<int32_t*>(extra + tok_bytes + vec_bytes);
    S1.p.out_tokens = tok1;
    S1.p.out_n = n1;
    S2.p.tokens = tok1;
    S2.p.dlen = len2;
    S2.p.stage = 1;
    S2.p.out_tokens = out_tokens;
    S2.p.out_n = out_n;
    rc = launch_verify(S1);
    if (rc) return rc;
    const hipError_t e = sv::launch_hispec_link(n1, len2, out_n_stage1, B, S1.stream);
    if (e != hipSuccess) return hip_fail(e, "kernel launch");
    return launch_verify(S2);
}

// Greedy verify: the statistics pass over the target rows with candidate
// lists (at T = 1, which only scales the list bins), then one workgroup per
// batch row for the argmaxes, the decision and the top-k.
int greedy_impl(const sv_logits* tl, const int32_t* draft_tokens, const int32_t* draft_len, int32_t k,
                int32_t* out_tokens, int32_t* out_n, int32_t* out_topk, void* stream_v) {
    if (!out_tokens || !out_n || (k > 0 && !out_topk)) return SV_EINVAL;
    if (k < 0 || k > sv::kMaxTopK) return SV_EINVAL;
    if (misaligned(out_tokens, 4) || misaligned(out_n, 4) || (out_topk && misaligned(out_topk, 4))) return SV_EALIGN;
    Setup S;
    int rc = prepare(tl, nullptr, draft_tokens, draft_len, 1.f, 1.f, 0, MODE_GREEDY, stream_v, S);
    if (rc) return rc;
    Params& p = S.p;
    p.out_tokens = out_tokens;
    p.out_n = out_n;
    p.topk = k;
    p.out_topk = out_topk;
    const hipStream_t stream = S.stream;
    rc = timed_launch(sv::KK_STATS, stream, [&](const sv::LaunchEvents& ev) {
        return sv::launch_greedy_stats(p, S.dtype, S.unroll, stream, ev);
    });
    if (rc) return rc;
    return timed_launch(sv::KK_RESAMPLE, stream,
                        [&](const sv::LaunchEvents& ev) { return sv::launch_greedy_rows(p, S.dtype, stream, ev); });
}

int smc_impl(const sv_logits* tl, const sv_logits* dl, const int32_t* draft_tokens, const double* logw_in,
             float temperature, double ess_fraction, uint64_t seed, int32_t* out_bonus, double* out_logw,
             int32_t* out_ancestor, double* out_ess, int32_t* out_resampled, void* stream_v) {
    if (!logw_in || !out_bonus || !out_logw || !out_ancestor || !out_ess || !out_resampled) return SV_EINVAL;
    if (misaligned(logw_in, 8) || misaligned(out_logw, 8) || misaligned(out_ess, 8) || misaligned(out_bonus, 4) ||
        misaligned(out_ancestor, 4) || misaligned(out_resampled, 4))
        return SV_EALIGN;
    if (std::isnan(ess_fraction)) return SV_EINVAL;
    Setup S;
    int rc = prepare(tl, dl, draft_tokens, nullptr, temperature, 1.f, seed, MODE_SMC, stream_v, S);
    if (rc) return rc;
    Params& p = S.p;
    p.out_tokens = out_bonus;
    p.ess_frac = ess_fraction;
    p.logw_in = logw_in;
    p.logw_out = out_logw;
    p.out_ancestor = out_ancestor;
    p.out_ess = out_ess;
    p.out_resampled = out_resampled;
    const hipStream_t stream = S.stream;
    rc = timed_launch(sv::KK_STATS, stream, [&](const sv::LaunchEvents& ev) {
        return sv::launch_stats(p, S.dtype, S.unroll, false, stream, ev);
    });
    if (rc) return rc;
    rc = timed_launch(sv::KK_RESAMPLE, stream,
                      [&](const sv::LaunchEvents& ev) { return sv::launch_smc_rows(p, S.dtype, stream, ev); });
    if (rc) return rc;
    return timed_launch(sv::KK_SMC, stream,
                        [&](const sv::LaunchEvents& ev) { return sv::launch_smc_resample(p, stream, ev); });
}

// Synthetic draft producer of the two-batch schedule: drafts and chunk
// records, then the tokens.  Its chunk records use the (device, stream)
// scratch like every other call on that stream.
int produce_impl(const sv_logits* tl, int32_t K, uint64_t seed, void* out, int64_t osb, int64_t osp,
                 int32_t* out_tokens, void* stream_v) {
    int rc = check_logits(tl);
    if (rc) return rc;
    if (!out || !out_tokens) return SV_EINVAL;
    const int E = tl->dtype == SV_BF16 ? 2 : 4;
    if (misaligned(out, E) || misaligned(out_tokens, 4)) return SV_EALIGN;
    if (osb < 0 || osp < 0) return SV_EINVAL;
    const int B = tl->B, V = tl->V;
    if (B <= 0 || V <= 0 || K < 1 || K > tl->P || B > (1 << 22) || V > (1 << 24)) return SV_ESHAPE;
    const int64_t groups = (static_cast<int64_t>(V) + 7) / 8;
    const int64_t per = static_cast<int64_t>(sv::kThreads) * sv::kProdU;
    const int nchp = static_cast<int>((groups + per - 1) / per);
    if (static_cast<int64_t>(B) * K * nchp >= (1ll << 31)) return SV_ESHAPE;
    const hipStream_t stream = static_cast<hipStream_t>(stream_v);
    void* base = nullptr;
    rc = get_scratch(stream, static_cast<size_t>(B) * K * nchp * 2 * sizeof(uint64_t), &base);
    if (rc) return rc;
    sv::ProduceParams p;
    std::memset(&p, 0, sizeof(p));
    p.tgt = static_cast<const uint8_t*>(tl->data);
    p.tsb = tl->stride_b;
    p.tsp = tl->stride_p;
    p.out = static_cast<uint8_t*>(out);
    p.osb = osb;
    p.osp = osp;
    p.tokens = out_tokens;
    p.rec = static_cast<uint64_t*>(base);
    p.B = B;
    p.K = K;
    p.V = V;
    p.nchp = nchp;
    p.k0 = static_cast<uint32_t>(seed);
    p.k1 = static_cast<uint32_t>(seed >> 32);
    p.tag = next_tag();
    const int dtype = tl->dtype == SV_BF16 ? sv::DT_BF16 : sv::DT_F32;
    rc = timed_launch(sv::KK_PRODUCE, stream,
                      [&](const sv::LaunchEvents& ev) { return sv::launch_produce(p, dtype, stream, ev); });
    if (rc) return rc;
    return timed_launch(sv::KK_PRODUCE, stream,
                        [&](const sv::LaunchEvents& ev) { return sv::launch_produce_tokens(p, stream, ev); });
}

// ---- the tree round ----

static_assert(SPECVERIFY_MAX_NODES == sv::kMaxNodes && SPECVERIFY_MAX_PAGES == sv::kMaxPages &&
                  SV_F16 == sv::kDTypeF16, "tree limits");

bool pow2_page(int ps) { return ps >= 1 && ps <= 1024 && (ps & (ps - 1)) == 0; }

// Strides of a tensor whose rows are read 16 bytes at a time, `size` along its
// axes; they come out in units of 16 bytes, 0 for an axis of one.
template <typename I>
int check_rows(const void* data, const int64_t* stride, const int32_t* size, int n, int elem, I* out) {
    if (!data) return SV_EINVAL;
    for (int i = 0; i < n; ++i)
        if (size[i] > 1 && stride[i] < 0) return SV_EINVAL;
    if (misaligned(data, 16)) return SV_EALIGN;
    for (int i = 0; i < n; ++i) {
        out[i] = 0;
        if (size[i] == 1) continue;
        if (stride[i] > (1ll << 40) || stride[i] / (16 / elem) > static_cast<int64_t>(std::numeric_limits<I>::max()))
            return SV_ESHAPE;
        if (stride[i] * elem % 16) return SV_EALIGN;
        out[i] = static_cast<I>(stride[i] / (16 / elem));
    }
    return SV_OK;
}

// Rows that are written must not fall together (from check_rows' strides): an
// axis longer than one with stride 0 is an expanded tensor.
template <typename I>
bool expanded(const I* stride, const int32_t* size, int n) {
    for (int i = 0; i < n; ++i)
        if (size[i] > 1 && stride[i] == 0) return true;
    return false;
}

// |scale| log2(e).  (-inf) times it has to stay -inf, and 0 times it 0: no zero, no denormal, not infinite.
float score_scale(float scale) {
    const float s = static_cast<float>(
        std::min(std::fabs(static_cast<double>(scale)) * 1.4426950408889634074, static_cast<double>(FLT_MAX)));
    return s < FLT_MIN ? FLT_MIN : s;
}

// How the attention's work is cut: rows and keys per workgroup tile by the
// query rows that share a key head, parts by the device's size.  64 sequences
// of 4096 rows, 8 key heads of 128, us with tiles of 32 / 64 / 128 rows: 24
// rows 201 / 210 / 221, 36 rows 237 / 211, 64 rows 241 / 212 / 230, 128 rows
// - / 266 / 237.
struct TreePlan {
    sv::TreeAttnShape s;
    int MT = 1, clusters = 1, merge = 0;
    size_t start_bytes = 0, total = 0;
};

int plan_tree(const sv_tree_attention* a, TreePlan& t) {
    if (!a) return SV_EINVAL;
    if (a->dtype != SV_BF16 && a->dtype != SV_F16) return SV_EDTYPE;
    if (a->B < 1 || a->B > 65536 || a->N < 1 || a->N > SPECVERIFY_MAX_NODES) return SV_ESHAPE;
    if (a->heads < 1 || a->kv_heads < 1 || a->heads > 1024 || a->heads % a->kv_heads) return SV_ESHAPE;
    if (a->dim < 8 || a->dim > 128 || a->dim % 8) return SV_ESHAPE;
    if (a->pages < 1 || !pow2_page(a->page_size) || a->width < 0) return SV_ESHAPE;
    if (static_cast<int64_t>(a->width) * a->page_size > (1ll << 28)) return SV_ESHAPE;
    const int rows = a->N * (a->heads / a->kv_heads);
    t.s.dp = a->dim <= 64 ? 64 : 128;
    t.s.rows = rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
    t.s.keys = t.s.rows == 32 ? 128 : 64;
    t.MT = (rows + t.s.rows - 1) / t.s.rows;
    const int64_t tasks = static_cast<int64_t>(a->B) * a->kv_heads;
    // a launch has fewer than 2^32 threads; several row tiles go in groups of eight parts
    if ((t.MT > 1 ? (tasks + 7) / 8 * 8 : tasks) * t.MT >= 1ll << 24) return SV_ESHAPE;
    const int64_t cap = static_cast<int64_t>(a->width) * a->page_size;
    const int64_t most = (cap + t.s.keys - 1) / t.s.keys + 1;  // tiles of one (sequence, key head)
    if (a->kv_heads * most > 1ll << 32) return SV_ESHAPE;  // the kernel counts a sequence's tiles in 32 bits
    // As many parts as workgroups are resident at once: 32 rows of 128 dimensions take
    // 128 KB of LDS, one workgroup per CU; else two.  As above with one and two parts per
    // CU: 24 rows 197 and 208 us, 64 rows 223 and 213, 128 rows 258 and 238.
    const int64_t blocks = (t.s.rows == 32 && t.s.dp == 128 ? 1ll : 2ll) * device_cus();
    if (most <= 4) {
        // So short that a part is a whole (sequence, key head) and nothing is joined: 64
        // sequences of 384 rows 35 us, divided and joined 34 + 4; one sequence of 384 rows 14
        // and 11 + 4, of 768 (more than four tiles) 17 and 11 + 4.
        t.merge = 0;
        t.clusters = static_cast<int>(tasks);
    } else {
        t.merge = 1;
        int64_t c = blocks / t.MT;
        if (c > tasks * most) c = tasks * most;
        t.clusters = static_cast<int>(c < 1 ? 1 : c);
        t.start_bytes = align256((static_cast<size_t>(a->B) + 1) * sizeof(int64_t));
        t.total = t.start_bytes +
                  static_cast<size_t>(t.clusters) * 2 * t.MT * t.s.rows * (t.s.dp + 2) * sizeof(float);
    }
    return SV_OK;
}

int tree_attention_impl(const sv_tree_attention* a, void* stream_v) {
    TreePlan t;
    int rc = plan_tree(a, t);
    if (rc) return rc;
    sv::TreeAttnParams p;
    std::memset(&p, 0, sizeof(p));
    if (!a->out || !a->len || !a->parent || (a->width > 0 && !a->table)) return SV_EINVAL;
    if (a->table_stride < 0 || a->window < 0 || a->sinks < 0 || !std::isfinite(a->scale)) return SV_EINVAL;
    const int32_t nodes[3] = {a->B, a->N, a->heads}, tree[3] = {a->B, a->N, a->kv_heads},
                  cache[3] = {a->pages, a->page_size, a->kv_heads};
    const struct {
        const void* data;
        const int64_t* stride;
        const int32_t* size;
        uint32_t* out;
    } rows[] = {{a->q, a->q_stride, nodes, p.qs},
                {a->k_tree, a->k_tree_stride, tree, p.kts},
                {a->v_tree, a->v_tree_stride, tree, p.vts},
                {a->k_cache, a->k_cache_stride, cache, p.kcs},
                {a->v_cache, a->v_cache_stride, cache, p.vcs},
                {a->out, a->out_stride, nodes, p.os}};
    for (const auto& r : rows) {
        rc = check_rows(r.data, r.stride, r.size, 3, 2, r.out);
        if (rc) return rc;
    }
    if (expanded(p.os, nodes, 3)) return SV_EINVAL;
    if (misaligned(a->table, 4) || misaligned(a->len, 4) || misaligned(a->parent, 4) ||
        (a->n_nodes && misaligned(a->n_nodes, 4)))
        return SV_EALIGN;
    if (t.total > 0) {
        if (!a->workspace) return SV_EINVAL;
        if (misaligned(a->workspace, 16)) return SV_EALIGN;
        if (a->workspace_bytes < 0 || static_cast<size_t>(a->workspace_bytes) < t.total) return SV_ETOOBIG;
    }
    p.q = static_cast<const uint8_t*>(a->q);
    p.kt = static_cast<const uint8_t*>(a->k_tree);
    p.vt = static_cast<const uint8_t*>(a->v_tree);
    p.kc = static_cast<const uint8_t*>(a->k_cache);
    p.vc = static_cast<const uint8_t*>(a->v_cache);
    p.out = static_cast<uint8_t*>(a->out);
    p.table = a->table;
    p.table_stride = a->table_stride;
    p.len = a->len;
    p.parent = a->parent;
    p.n_nodes = a->n_nodes;
    p.B = a->B;
    p.N = a->N;
    p.Hkv = a->kv_heads;
    p.G = a->heads / a->kv_heads;
    p.D = a->dim;
    p.pages = a->pages;
    p.width = a->width;
    p.ps_shift = __builtin_ctz(static_cast<unsigned>(a->page_size));
    // beyond every length and depth both mean everything; the kernel subtracts row numbers from them
    p.window = std::min(a->window, 1 << 29);
    p.sinks = std::min(a->sinks, 1 << 29);
    p.scale2 = score_scale(a->scale);
    p.flip = a->scale < 0.f ? 1 : 0;
    p.MT = t.MT;
    p.clusters = t.clusters;
    p.merge = t.merge;
    if (t.merge) {
        p.start = static_cast<int64_t*>(a->workspace);
        p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a->workspace) + t.start_bytes);
    }
    const int dtype = a->dtype == SV_BF16 ? static_cast<int>(sv::DT_BF16) : sv::kDTypeF16;
    const hipStream_t stream = static_cast<hipStream_t>(stream_v);
    rc = timed_launch(sv::KK_TREE_ATTN, stream,
                      [&](const sv::LaunchEvents& ev) { return sv::launch_tree_attn(p, t.s, dtype, stream, ev); });
    if (rc || !t.merge) return rc;
    return timed_launch(sv::KK_TREE_MERGE, stream,
                        [&](const sv::LaunchEvents& ev) { return sv::launch_tree_merge(p, t.s, dtype, stream, ev); });
}

// Workgroups per sequence: as many as give every CU one (each fills it), while
// a range keeps at least one block of ids (256 float32, 512 bfloat16).  A team
// pays for the launch that clears its workspace where a sequence makes several
// passes: one sequence of V = 128256 (float32, trees of two drawn children) 19
// us with sixteen and 30 with one, 64 of them 37 with four and 63 with one.
// Without draft probabilities there is one pass (one sequence: 16 and 13 us).
// From 65 sequences on there is no team: with one / two / three workgroups each,
// trees of 16 drawn nodes take 44 / 38 / 37 us (65 sequences), 56 / 46 / 47 (96),
// 66 / 55 / 64 (128), 73 / 73 / 82 (192), in bfloat16 41 / 35 / 32, 47 / 39 / 39,
// 47 / 42 / 51, 50 / 56 / 62: teams of two up to 128 would gain an eighth.
int verify_team(int B, int V, int dtype, bool draft) {
    if (!draft) return 1;
    int team = device_cus() / B;
    const int most = V / (sv::kVerifyWaves * (dtype == SV_BF16 ? 512 : 256));
    team = std::min(std::min(team, most), sv::kMaxTeam);
    return team < 4 ? 1 : team;
}

int64_t verify_workspace(int64_t B, int64_t N, int team) {
    return team > 1 ? B * (N + 2) * team * sv::kVerifyWaves * static_cast<int64_t>(sizeof(uint64_t)) : 0;
}

int verify_tree_impl(const sv_logits* tp, const sv_logits* dp, const int32_t* tokens, const int32_t* parent,
                     const int32_t* n_nodes, const float* u_accept, const float* u_final, int32_t* out_tokens,
                     int32_t* out_nodes, int32_t* out_n, void* ws, int64_t ws_bytes, void* stream_v) {
    int rc = check_logits(tp);
    if (rc) return rc;
    if (dp) {
        rc = check_logits(dp);
        if (rc) return rc;
    }
    if (!tokens || !parent || !u_accept || !u_final || !out_tokens || !out_nodes || !out_n) return SV_EINVAL;
    if (misaligned(tokens, 4) || misaligned(parent, 4) || (n_nodes && misaligned(n_nodes, 4)) ||
        misaligned(u_accept, 4) || misaligned(u_final, 4) || misaligned(out_tokens, 4) || misaligned(out_nodes, 4) ||
        misaligned(out_n, 4))
        return SV_EALIGN;
    if (dp && dp->dtype != tp->dtype) return SV_EDTYPE;
    const int B = tp->B, N = tp->P, V = tp->V;
    if (B < 1 || B >= 1 << 22 || N < 1 || N > SPECVERIFY_MAX_NODES || V < 1 || V > SPECVERIFY_MAX_V) return SV_ESHAPE;
    // another workgroup of the team may still read the inputs when the first one writes
    for (const int32_t* in : {tokens, parent, n_nodes})
        if (in && (in == out_tokens || in == out_nodes || in == out_n)) return SV_EINVAL;
    if (out_tokens == out_nodes) return SV_EINVAL;
    if (dp && (dp->B != B || dp->V != V || dp->P < 1 || dp->P > N)) return SV_ESHAPE;
    const int team = verify_team(B, V, tp->dtype, dp != nullptr);
    if (team > 1) {
        if (!ws) return SV_EINVAL;
        if (misaligned(ws, 8)) return SV_EALIGN;
        if (ws_bytes < verify_workspace(B, N, team)) return SV_ETOOBIG;
    }
    sv::TreeVerifyParams p;
    std::memset(&p, 0, sizeof(p));
    p.tgt = static_cast<const uint8_t*>(tp->data);
    p.tsb = tp->stride_b;
    p.tsp = tp->stride_p;
    if (dp) {
        p.dft = static_cast<const uint8_t*>(dp->data);
        p.dsb = dp->stride_b;
        p.dsp = dp->stride_p;
        p.P = dp->P;
    }
    p.tokens = tokens;
    p.parent = parent;
    p.n_nodes = n_nodes;
    p.u_accept = u_accept;
    p.u_final = u_final;
    p.out_tokens = out_tokens;
    p.out_nodes = out_nodes;
    p.out_n = out_n;
    p.B = B;
    p.N = N;
    p.V = V;
    p.team = team;
    p.passes = N + 2;
    // SPECVERIFY_VERIFY_LOOKS replaces it (tests: with 0 every workgroup sums the rows by itself)
    p.looks = std::min(std::max(env_int("SPECVERIFY_VERIFY_LOOKS", 16), 0), 64);
    p.rec = static_cast<uint64_t*>(ws);
    const int dtype = tp->dtype == SV_BF16 ? sv::DT_BF16 : sv::DT_F32;
    const hipStream_t stream = static_cast<hipStream_t>(stream_v);
    if (team > 1) {
        rc = timed_launch(sv::KK_VERIFY_CLEAR, stream,
                          [&](const sv::LaunchEvents& ev) { return sv::launch_verify_clear(p, stream, ev); });
        if (rc) return rc;
    }
    return timed_launch(sv::KK_TREE_VERIFY, stream,
                        [&](const sv::LaunchEvents& ev) { return sv::launch_tree_verify(p, dtype, stream, ev); });
}

// Workspace of a commit or fork: the plan, its own words, the new pages.
int64_t cache_workspace(int64_t B, int64_t N, int64_t page_size) {
    const int64_t fresh = N > 0 ? (N + page_size - 1) / page_size + 1 : 1;
    return 4 * B * (sv::kPlanWords + sv::kPlanSpare + fresh);
}

int cache_impl(const sv_cache* c, const void* kt, const void* vt, const int64_t* kts, const int64_t* vts, int32_t N,
               const int32_t* nodes, const int32_t* n_accepted, const int32_t* ancestor, bool fork,
               int32_t* out_table, int64_t out_stride, int32_t* out_len, int32_t* out_status, void* ws,
               int64_t ws_bytes, void* stream_v) {
    if (!c) return SV_EINVAL;
    if (c->dtype != SV_F32 && c->dtype != SV_BF16 && c->dtype != SV_F16) return SV_EDTYPE;
    const int elem = c->dtype == SV_F32 ? 4 : 2;
    if (c->B < 1 || c->B > 65534 || c->layers < 1 || c->layers > 65534 || c->heads < 1 || c->heads > 4096 ||
        c->dim < 1 || c->dim > 65536 || c->pages < 1 || c->pages > SPECVERIFY_MAX_PAGES || !pow2_page(c->page_size) ||
        c->width < 1 || static_cast<int64_t>(c->width) * c->page_size > (1ll << 28))
        return SV_ESHAPE;
    if (!fork && (N < 1 || N > SPECVERIFY_MAX_NODES)) return SV_ESHAPE;
    // 16-byte vectors a sequence moves per layer: the copies count them in 32 bits
    if (static_cast<int64_t>(c->heads) * c->dim * elem / 16 * (fork ? c->page_size : N) > (1ll << 30)) return SV_ESHAPE;
    if (!c->table || !c->len || !out_table || !out_len || !out_status || !ws) return SV_EINVAL;
    if (fork ? !ancestor : !n_accepted) return SV_EINVAL;
    if (c->table_stride < 0 || out_stride < c->width) return SV_EINVAL;
    // a fork permutes rows; a commit may run in place, row on row
    if (fork && (out_table == c->table || out_len == c->len)) return SV_EINVAL;
    if (!fork && out_table == c->table && out_stride != c->table_stride) return SV_EINVAL;
    if (misaligned(c->table, 4) || misaligned(c->len, 4) || misaligned(out_table, 4) || misaligned(out_len, 4) ||
        misaligned(out_status, 4) || misaligned(ws, 4) || (nodes && misaligned(nodes, 4)) ||
        (n_accepted && misaligned(n_accepted, 4)) || (ancestor && misaligned(ancestor, 4)))
        return SV_EALIGN;
    if (static_cast<int64_t>(c->dim) * elem % 16) return SV_EALIGN;
    sv::CacheParams p;
    std::memset(&p, 0, sizeof(p));
    const int64_t unit = 16 / elem;
    const int32_t size[4] = {c->layers, c->pages, c->page_size, c->heads}, tree[4] = {c->layers, c->B, N, c->heads};
    int rc = check_rows(c->k, c->k_stride, size, 4, elem, p.ks);
    if (!rc) rc = check_rows(c->v, c->v_stride, size, 4, elem, p.vs);
    if (!rc && (expanded(p.ks, size, 4) || expanded(p.vs, size, 4))) rc = SV_EINVAL;
    if (!rc && !fork) {
        if (!kts || !vts) return SV_EINVAL;
        rc = check_rows(kt, kts, tree, 4, elem, p.kts);
        if (!rc) rc = check_rows(vt, vts, tree, 4, elem, p.vts);
    }
    if (rc) return rc;
    if (ws_bytes < cache_workspace(c->B, fork ? 0 : N, c->page_size)) return SV_ETOOBIG;
    p.k = static_cast<uint8_t*>(c->k);
    p.v = static_cast<uint8_t*>(c->v);
    p.kt = static_cast<const uint8_t*>(kt);
    p.vt = static_cast<const uint8_t*>(vt);
    p.layers = c->layers;
    p.pages = c->pages;
    p.ps_shift = __builtin_ctz(static_cast<unsigned>(c->page_size));
    p.heads = c->heads;
    p.vec = static_cast<int>(c->dim / unit);
    p.table = c->table;
    p.len = c->len;
    p.out_table = out_table;
    p.out_len = out_len;
    p.status = out_status;
    p.table_stride = c->table_stride;
    p.out_stride = out_stride;
    p.B = c->B;
    p.N = N;
    p.width = c->width;
    p.nodes = nodes;
    p.n_accepted = n_accepted;
    p.ancestor = ancestor;
    p.fork = fork ? 1 : 0;
    p.plan = static_cast<int32_t*>(ws);
    const hipStream_t stream = static_cast<hipStream_t>(stream_v);
    rc = timed_launch(sv::KK_CACHE_PLAN, stream,
                      [&](const sv::LaunchEvents& ev) { return sv::launch_cache_plan(p, stream, ev); });
    if (rc) return rc;
    return timed_launch(sv::KK_CACHE_COPY, stream,
                        [&](const sv::LaunchEvents& ev) { return sv::launch_cache_copy(p, stream, ev); });
}

// How the latent attention's work is cut: rows per workgroup tile by the query
// rows that share a sequence's cache rows, parts by the device's size.
struct LatentPlan {
    sv::LatentShape s;
    int MT = 1, clusters = 1, merge = 0;
    size_t start_bytes = 0, total = 0;
};

int plan_latent(const sv_latent_attention* a, LatentPlan& t) {
    if (!a) return SV_EINVAL;
    if (a->dtype != SV_BF16 && a->dtype != SV_F16) return SV_EDTYPE;
    if (a->B < 1 || a->B > 65536 || a->N < 1 || a->N > SPECVERIFY_MAX_NODES) return SV_ESHAPE;
    if (a->heads < 1 || a->heads > 1024) return SV_ESHAPE;
    if (a->dim < 8 || a->dim > SPECVERIFY_MAX_LATENT || a->dim % 8) return SV_ESHAPE;
    if (a->dim_v < 8 || a->dim_v > a->dim || a->dim_v > 512 || a->dim_v % 8) return SV_ESHAPE;
    if (a->pages < 1 || !pow2_page(a->page_size) || a->width < 0) return SV_ESHAPE;
    if (static_cast<int64_t>(a->width) * a->page_size > (1ll << 28)) return SV_ESHAPE;
    const int rows = a->N * a->heads;
    t.s.wide = a->dim > 320 || a->dim_v > 256;
    // 64 rows share a tile's staging where there are that many (64 x 128: 90 us for 121 with 32; 32 x 256:
    // 136 for 190); up to 32 half the products would be of nothing
    t.s.rows = rows <= 32 ? 32 : 64;
    t.MT = (rows + t.s.rows - 1) / t.s.rows;
    // a launch has fewer than 2^32 threads
    if ((static_cast<int64_t>(a->B) + 7) / 8 * 8 * t.MT >= 1ll << 23) return SV_ESHAPE;
    const int64_t cap = static_cast<int64_t>(a->width) * a->page_size;
    const int64_t most = (cap + 31) / 32 + (a->N + 31) / 32;  // tiles of one sequence
    if (most <= 4) {
        t.merge = 0;
        t.clusters = a->B;
    } else {
        t.merge = 1;
        int64_t c = device_cus() / t.MT;
        if (c > a->B * most) c = a->B * most;
        t.clusters = static_cast<int>(c < 1 ? 1 : c);
        t.start_bytes = align256((static_cast<size_t>(a->B) + 1) * sizeof(int64_t));
        t.total = t.start_bytes + static_cast<size_t>(t.clusters) * 2 * t.MT * t.s.rows *
                                      (sv::latent_dv(t.s.wide) + 2) * sizeof(float);
    }
    return SV_OK;
}

int latent_attention_impl(const sv_latent_attention* a, void* stream_v) {
    LatentPlan t;
    int rc = plan_latent(a, t);
    if (rc) return rc;
    sv::LatentParams p;
    std::memset(&p, 0, sizeof(p));
    if (!a->out || !a->len || (a->width > 0 && !a->table)) return SV_EINVAL;
    if (a->table_stride < 0 || !std::isfinite(a->scale)) return SV_EINVAL;
    const int32_t heads[3] = {a->B, a->N, a->heads}, nodes[2] = {a->B, a->N}, cache[2] = {a->pages, a->page_size};
    rc = check_rows(a->q, a->q_stride, heads, 3, 2, p.qs);
    if (!rc) rc = check_rows(a->rows, a->rows_stride, nodes, 2, 2, p.nws);
    if (!rc) rc = check_rows(a->cache, a->cache_stride, cache, 2, 2, p.kcs);
    if (!rc) rc = check_rows(a->out, a->out_stride, heads, 3, 2, p.os);
    if (rc) return rc;
    if (expanded(p.os, heads, 3)) return SV_EINVAL;
    if (misaligned(a->table, 4) || misaligned(a->len, 4) || (a->parent && misaligned(a->parent, 4)) ||
        (a->n_nodes && misaligned(a->n_nodes, 4)))
        return SV_EALIGN;
    if (t.total > 0) {
        if (!a->workspace) return SV_EINVAL;
        if (misaligned(a->workspace, 16)) return SV_EALIGN;
        if (a->workspace_bytes < 0 || static_cast<size_t>(a->workspace_bytes) < t.total) return SV_ETOOBIG;
    }
    p.q = static_cast<const uint8_t*>(a->q);
    p.nw = static_cast<const uint8_t*>(a->rows);
    p.kc = static_cast<const uint8_t*>(a->cache);
    p.out = static_cast<uint8_t*>(a->out);
    p.table = a->table;
    p.table_stride = a->table_stride;
    p.len = a->len;
    p.parent = a->parent;
    p.n_nodes = a->n_nodes;
    p.B = a->B;
    p.N = a->N;
    p.H = a->heads;
    p.C = a->dim;
    p.dv = a->dim_v;
    p.pages = a->pages;
    p.width = a->width;
    p.ps_shift = __builtin_ctz(static_cast<unsigned>(a->page_size));
    p.scale2 = score_scale(a->scale);
    p.flip = a->scale < 0.f ? 1 : 0;
    p.MT = t.MT;
    p.clusters = t.clusters;
    p.merge = t.merge;
    if (t.merge) {
        p.start = static_cast<int64_t*>(a->workspace);
        p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a->workspace) + t.start_bytes);
    }
    const int dtype = a->dtype == SV_BF16 ? static_cast<int>(sv::DT_BF16) : sv::kDTypeF16;
    const hipStream_t stream = static_cast<hipStream_t>(stream_v);
    rc = timed_launch(sv::KK_LATENT_ATTN, stream,
                      [&](const sv::LaunchEvents& ev) { return sv::launch_latent_attn(p, t.s, dtype, stream, ev); });
    if (rc || !t.merge) return rc;
    return timed_launch(sv::KK_LATENT_JOIN, stream,
                        [&](const sv::LaunchEvents& ev) { return sv::launch_latent_join(p, t.s, dtype, stream, ev); });
}

int half_type(int32_t dtype) { return dtype == SV_BF16 ? static_cast<int>(sv::DT_BF16) : sv::kDTypeF16; }

int head_product_impl(const sv_head_product* a, void* stream_v) {
    if (!a) return SV_EINVAL;
    if (a->dtype != SV_BF16 && a->dtype != SV_F16) return SV_EDTYPE;
    if (a->T < 0 || a->T > 1 << 24 || a->heads < 1 || a->heads > 1024) return SV_ESHAPE;
    if (a->K < 8 || a->K > 65536 || a->K % 8 || a->M < 8 || a->M > 65536 || a->M % 8) return SV_ESHAPE;
    sv::ProductParams p;
    std::memset(&p, 0, sizeof(p));
    const int32_t tokens[2] = {a->T, a->heads}, rows[2] = {a->heads, a->M};
    if (a->T > 0) {
        int rc = check_rows(a->x, a->x_stride, tokens, 2, 2, p.xs);
        if (!rc) rc = check_rows(a->w, a->w_stride, rows, 2, 2, p.ws);
        if (!rc) rc = check_rows(a->out, a->out_stride, tokens, 2, 2, p.os);
        if (rc) return rc;
        if (expanded(p.os, tokens, 2)) return SV_EINVAL;
    }
    p.x = static_cast<const uint8_t*>(a->x);
    p.w = static_cast<const uint8_t*>(a->w);
    p.out = static_cast<uint8_t*>(a->out);
    p.T = a->T;
    p.H = a->heads;
    p.M = a->M;
    p.K = a->K;
    // up to 32 tokens a tile of 32: 128 heads 5.7 us for 7.0 with 128; 1024 tokens 43 for 59 with 32
    p.tt = a->T <= 32 ? 32 : 128;
    // a launch has fewer than 2^32 threads
    if (static_cast<int64_t>((p.M + 127) / 128) * ((p.T + p.tt - 1) / p.tt) * p.H >= (1ll << 24) - 8) return SV_ESHAPE;
    if (a->T == 0) return SV_OK;
    const hipStream_t stream = static_cast<hipStream_t>(stream_v);
    return timed_launch(sv::KK_PRODUCT, stream, [&](const sv::LaunchEvents& ev) {
        return sv::launch_product(p, half_type(a->dtype), stream, ev);
    });
}

// The workspace of a prompt call: places, flags, keys, values and second parts of the line.
struct PromptPlan {
    size_t odd, sizes, power, there, k, v, pe, total;
};

int plan_prompt(const sv_latent_prompt* a, PromptPlan& t) {
    if (!a) return SV_EINVAL;
    if (a->dtype != SV_BF16 && a->dtype != SV_F16) return SV_EDTYPE;
    if (a->B < 1 || a->B > 65536 || a->T < 0 || a->T > 1 << 24 || a->heads < 1 || a->heads > 1024) return SV_ESHAPE;
    if (a->dim_k < 8 || a->dim_k > 128 || a->dim_k % 8 || a->dim_p < 0 || a->dim_p > 64 || a->dim_p % 8 ||
        a->dim_v < 8 || a->dim_v > 128 || a->dim_v % 8)
        return SV_ESHAPE;
    if (a->latent < 8 || a->latent % 8 || a->latent + a->dim_p > SPECVERIFY_MAX_LATENT) return SV_ESHAPE;
    if (a->pages < 1 || !pow2_page(a->page_size) || a->width < 0) return SV_ESHAPE;
    if (static_cast<int64_t>(a->width) * a->page_size > (1ll << 28)) return SV_ESHAPE;
    if (a->rows < 0 || a->rows > 1 << 26) return SV_ESHAPE;
    // launches have fewer than 2^32 threads
    const int64_t lines = (static_cast<int64_t>(a->rows) + 127) / 128;
    const int64_t tiles = a->T / sv::kPromptRows + std::min(a->B, a->T);
    const int64_t out = (a->heads * a->dim_k + 127) / 128 + (a->heads * a->dim_v + 127) / 128;
    if (lines * out >= (1ll << 24) - 8 || tiles * a->heads >= (1ll << 24) - 8) return SV_ESHAPE;
    const size_t rows = static_cast<size_t>(lines) * 128;
    t.odd = align256((static_cast<size_t>(a->B) + 1) * 2 * sizeof(int64_t));
    t.sizes = t.odd + 256;
    t.power = align256(t.sizes + static_cast<size_t>(a->heads) * a->rows * sv::kSizeParts * sizeof(int16_t));
    t.there = align256(t.power + static_cast<size_t>(a->heads) * a->rows * sizeof(int16_t));
    t.k = align256(t.there + rows * sizeof(int32_t));
    t.v = align256(t.k + static_cast<size_t>(a->heads) * a->rows * a->dim_k * 2);
    t.pe = align256(t.v + static_cast<size_t>(a->heads) * a->rows * a->dim_v * 2);
    t.total = align256(t.pe + rows * a->dim_p * 2);
    return SV_OK;
}

int latent_prompt_impl(const sv_latent_prompt* a, void* stream_v) {
    PromptPlan t;
    int rc = plan_prompt(a, t);
    if (rc) return rc;
    if (!a->len || !a->q_start || (a->width > 0 && !a->table)) return SV_EINVAL;
    if (a->table_stride < 0 || !std::isfinite(a->scale)) return SV_EINVAL;
    sv::PromptParams p;
    std::memset(&p, 0, sizeof(p));
    const int32_t tokens[2] = {a->T, a->heads}, cache[2] = {a->pages, a->page_size}, wk[2] = {a->heads, a->dim_k},
                  wv[2] = {a->heads, a->dim_v};
    if (a->T > 0) {
        rc = check_rows(a->q, a->q_stride, tokens, 2, 2, p.qs);
        if (!rc) rc = check_rows(a->out, a->out_stride, tokens, 2, 2, p.os);
        if (!rc && expanded(p.os, tokens, 2)) rc = SV_EINVAL;
    }
    if (!rc) rc = check_rows(a->cache, a->cache_stride, cache, 2, 2, p.kcs);
    if (!rc) rc = check_rows(a->w_k, a->w_k_stride, wk, 2, 2, p.wks);
    if (!rc) rc = check_rows(a->w_v, a->w_v_stride, wv, 2, 2, p.wvs);
    if (rc) return rc;
    if (misaligned(a->table, 4) || misaligned(a->len, 4) || misaligned(a->q_start, 4)) return SV_EALIGN;
    if (!a->workspace) return SV_EINVAL;
    if (misaligned(a->workspace, 16)) return SV_EALIGN;
    if (a->workspace_bytes < 0 || static_cast<size_t>(a->workspace_bytes) < t.total) return SV_ETOOBIG;
    if (a->T == 0) return SV_OK;
    p.q = static_cast<const uint8_t*>(a->q);
    p.kc = static_cast<const uint8_t*>(a->cache);
    p.wk = static_cast<const uint8_t*>(a->w_k);
    p.wv = static_cast<const uint8_t*>(a->w_v);
    p.out = static_cast<uint8_t*>(a->out);
    p.table = a->table;
    p.len = a->len;
    p.q_start = a->q_start;
    p.table_stride = a->table_stride;
    p.T = a->T;
    p.B = a->B;
    p.H = a->heads;
    p.dn = a->dim_k;
    p.dr = a->dim_p;
    p.dv = a->dim_v;
    p.R = a->latent;
    p.rows = a->rows;
    p.pages = a->pages;
    p.width = a->width;
    p.ps_shift = __builtin_ctz(static_cast<unsigned>(a->page_size));
    p.scale2 = score_scale(a->scale);
    p.flip = a->scale < 0.f ? 1 : 0;
    p.cus = device_cus();
    uint8_t* const ws = static_cast<uint8_t*>(a->workspace);
    p.plan = reinterpret_cast<int64_t*>(ws);
    p.odd = reinterpret_cast<int32_t*>(ws + t.odd);
    p.sizes = reinterpret_cast<int16_t*>(ws + t.sizes);
    p.power = reinterpret_cast<int16_t*>(ws + t.power);
    p.there = reinterpret_cast<int32_t*>(ws + t.there);
    p.k = ws + t.k;
    p.v = ws + t.v;
    p.pe = ws + t.pe;
    const int dtype = half_type(a->dtype);
    const hipStream_t stream = static_cast<hipStream_t>(stream_v);
    rc = timed_launch(sv::KK_PROMPT_PLAN, stream,
                      [&](const sv::LaunchEvents& ev) { return sv::launch_prompt_plan(p, stream, ev); });
    for (const bool again : {false, true})
        if (!rc && a->rows > 0)
            rc = timed_launch(sv::KK_PROMPT_EXPAND + again, stream, [&](const sv::LaunchEvents& ev) {
                return sv::launch_prompt_expand(p, dtype, again, stream, ev);
            });
    if (rc) return rc;
    return timed_launch(sv::KK_PROMPT_ATTN, stream,
                        [&](const sv::LaunchEvents& ev) { return sv::launch_prompt_attn(p, dtype, stream, ev); });
}

static_assert(SPECVERIFY_MAX_BEAMS == sv::kMaxBeams, "beam limit");

// Runs of 2048 ids in a chunk of a row: four, or one where those would not fill the device.  256
// rows of 128256 ids: 49 us with four, 60 with one (more lists to select from); four such rows: 15.5
// with four, 14.4 with one.
int beam_runs(int64_t rows, int V) { return rows * ((V + 8191) / 8192) < 2 * device_cus() ? 1 : 4; }

int64_t beam_workspace(int64_t rows, int W, int V) {
    const int64_t ids = 2048 * beam_runs(rows, V), chunks = (V + ids - 1) / ids;
    return align256(rows * chunks * sizeof(sv::BeamChunk)) + rows * chunks * W * sizeof(uint64_t);
}

int check_beams(int B, int W, int V) {
    return B < 1 || W < 1 || W > SPECVERIFY_MAX_BEAMS || static_cast<int64_t>(B) * W > 65535 || V < 1 || V > 1 << 24
               ? SV_ESHAPE
               : SV_OK;
}

int beam_select_impl(const sv_logits* l, const float* scores, const int32_t* finished, int32_t end, int32_t* out_tokens,
                     int32_t* out_ancestor, float* out_scores, int32_t* out_finished, void* ws, int64_t ws_bytes,
                     void* stream_v) {
    int rc = check_logits(l);
    if (rc) return rc;
    if (!scores || !out_tokens || !out_ancestor || !out_scores || !out_finished || !ws) return SV_EINVAL;
    if (misaligned(scores, 4) || (finished && misaligned(finished, 4)) || misaligned(out_tokens, 4) ||
        misaligned(out_ancestor, 4) || misaligned(out_scores, 4) || misaligned(out_finished, 4) || misaligned(ws, 8))
        return SV_EALIGN;
    rc = check_beams(l->B, l->P, l->V);
    if (rc) return rc;
    if (end < -1 || end >= l->V || (finished && end < 0)) return SV_EINVAL;
    if (out_scores == scores || (finished && out_finished == finished)) return SV_EINVAL;
    const int64_t rows = static_cast<int64_t>(l->B) * l->P;
    if (ws_bytes < beam_workspace(rows, l->P, l->V)) return SV_ETOOBIG;
    sv::BeamParams p;
    std::memset(&p, 0, sizeof(p));
    p.logits = static_cast<const uint8_t*>(l->data);
    p.sb = l->stride_b;
    p.sw = l->stride_p;
    p.scores = scores;
    p.finished = finished;
    p.out_tokens = out_tokens;
    p.out_ancestor = out_ancestor;
    p.out_finished = out_finished;
    p.out_scores = out_scores;
    p.B = l->B;
    p.W = l->P;
    p.V = l->V;
    p.end = end;
    p.runs = beam_runs(rows, l->V);
    p.chunks = (l->V + 2048 * p.runs - 1) / (2048 * p.runs);
    p.rec = static_cast<sv::BeamChunk*>(ws);
    p.list = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(ws) + align256(rows * p.chunks * sizeof(sv::BeamChunk)));
    const int dtype = l->dtype == SV_BF16 ? sv::DT_BF16 : sv::DT_F32;
    const hipStream_t stream = static_cast<hipStream_t>(stream_v);
    rc = timed_launch(sv::KK_BEAM_STATS, stream,
                      [&](const sv::LaunchEvents& ev) { return sv::launch_beam_stats(p, dtype, stream, ev); });
    if (rc) return rc;
    return timed_launch(sv::KK_BEAM_SELECT, stream,
                        [&](const sv::LaunchEvents& ev) { return sv::launch_beam_select(p, dtype, stream, ev); });
}

int beam_reorder_impl(const void* src, int64_t src_stride, void* dst, int64_t dst_stride, int64_t row_bytes,
                      int32_t rows, const int32_t* ancestor, void* stream_v) {
    if (rows < 1 || rows > 65535 || row_bytes < 0 || row_bytes > 1ll << 40) return SV_ESHAPE;
    if (src_stride < 0 || src_stride > 1ll << 44 || dst_stride > 1ll << 44) return SV_EINVAL;
    if (rows > 1 && dst_stride < row_bytes) return SV_EINVAL;
    if (!ancestor || (row_bytes > 0 && (!src || !dst || src == dst))) return SV_EINVAL;
    if (misaligned(ancestor, 4)) return SV_EALIGN;
    if (row_bytes == 0) return SV_OK;
    sv::ReorderParams p;
    p.src = static_cast<const uint8_t*>(src);
    p.dst = static_cast<uint8_t*>(dst);
    p.ancestor = ancestor;
    p.src_stride = src_stride;
    p.dst_stride = rows > 1 ? dst_stride : 0;
    p.bytes = row_bytes;
    p.rows = rows;
    const hipStream_t stream = static_cast<hipStream_t>(stream_v);
    return timed_launch(sv::KK_BEAM_REORDER, stream,
                        [&](const sv::LaunchEvents& ev) { return sv::launch_reorder(p, stream, ev); });
}

int64_t reserve_workspace(int64_t B, int64_t page_size, int64_t rows) {
    return 4 * (B * sv::kReserveWords + rows / page_size + std::min(B, rows));
}

int check_reserve(int32_t B, int32_t page_size, int32_t rows) {
    return B < 1 || B > 65534 || !pow2_page(page_size) || rows < 0 || rows > 1 << 30 ? SV_ESHAPE : SV_OK;
}

int cache_reserve_impl(const int32_t* table, int64_t table_stride, const int32_t* len, const int32_t* n_new, int32_t B,
                       int32_t width, int32_t pages, int32_t page_size, int32_t rows, int32_t* out_table,
                       int64_t out_stride, int32_t* out_len, int32_t* out_start, int32_t* out_slots,
                       int32_t* out_position, int32_t* out_status, void* ws, int64_t ws_bytes, void* stream_v) {
    int rc = check_reserve(B, page_size, rows);
    if (rc) return rc;
    if (pages < 1 || pages > SPECVERIFY_MAX_PAGES || width < 1 || static_cast<int64_t>(width) * page_size > (1ll << 28) ||
        B * (static_cast<int64_t>(width) / 64 + 1) >= 1ll << 31)
        return SV_ESHAPE;
    if (!table || !len || !n_new || !out_table || !out_len || !out_start || !out_status || !ws ||
        (rows > 0 && (!out_slots || !out_position)))
        return SV_EINVAL;
    if (table_stride < 0 || out_stride < width || (out_table == table && out_stride != table_stride)) return SV_EINVAL;
    for (const void* q : {static_cast<const void*>(table), static_cast<const void*>(len),
                          static_cast<const void*>(n_new), static_cast<const void*>(out_table),
                          static_cast<const void*>(out_len), static_cast<const void*>(out_start),
                          static_cast<const void*>(out_slots), static_cast<const void*>(out_position),
                          static_cast<const void*>(out_status), static_cast<const void*>(ws)})
        if (misaligned(q, 4)) return SV_EALIGN;
    if (ws_bytes < reserve_workspace(B, page_size, rows)) return SV_ETOOBIG;
    sv::ReserveParams p;
    std::memset(&p, 0, sizeof(p));
    p.table = table;
    p.len = len;
    p.n_new = n_new;
    p.table_stride = table_stride;
    p.out_stride = out_stride;
    p.out_table = out_table;
    p.out_len = out_len;
    p.start = out_start;
    p.slots = out_slots;
    p.position = out_position;
    p.status = out_status;
    p.B = B;
    p.width = width;
    p.pages = pages;
    p.ps_shift = __builtin_ctz(static_cast<unsigned>(page_size));
    p.rows = rows;
    p.plan = static_cast<int32_t*>(ws);
    const hipStream_t stream = static_cast<hipStream_t>(stream_v);
    rc = timed_launch(sv::KK_RESERVE_PLAN, stream,
                      [&](const sv::LaunchEvents& ev) { return sv::launch_reserve_plan(p, stream, ev); });
    if (rc) return rc;
    return timed_launch(sv::KK_RESERVE_WRITE, stream,
                        [&](const sv::LaunchEvents& ev) { return sv::launch_reserve_write(p, stream, ev); });
}

int cache_write_impl(const sv_cache_rows* a, void* stream_v) {
    if (!a) return SV_EINVAL;
    if (a->dtype != SV_F32 && a->dtype != SV_BF16 && a->dtype != SV_F16) return SV_EDTYPE;
    const int elem = a->dtype == SV_F32 ? 4 : 2;
    if (a->pages < 1 || a->pages > SPECVERIFY_MAX_PAGES || !pow2_page(a->page_size) || a->T < 0 || a->T > 1 << 28 ||
        a->dim_a < 1 || a->dim_a > 65536 || a->dim_b < 0 || a->dim_b > 65536)
        return SV_ESHAPE;
    if (static_cast<int64_t>(a->dim_a) * elem % 16 || static_cast<int64_t>(a->dim_b) * elem % 16) return SV_EALIGN;
    if (a->T == 0) return SV_OK;
    if (!a->slots) return SV_EINVAL;
    if (misaligned(a->slots, 4)) return SV_EALIGN;
    sv::WriteParams p;
    std::memset(&p, 0, sizeof(p));
    const int32_t cache[2] = {a->pages, a->page_size}, tokens[1] = {a->T};
    int rc = check_rows(a->cache, a->cache_stride, cache, 2, elem, p.cs);
    if (!rc && expanded(p.cs, cache, 2)) rc = SV_EINVAL;
    if (!rc) rc = check_rows(a->a, &a->a_stride, tokens, 1, elem, &p.as);
    if (!rc && a->dim_b > 0) rc = check_rows(a->b, &a->b_stride, tokens, 1, elem, &p.bs);
    if (rc) return rc;
    p.cache = static_cast<uint8_t*>(a->cache);
    p.a = static_cast<const uint8_t*>(a->a);
    p.b = static_cast<const uint8_t*>(a->b);
    p.slots = a->slots;
    p.T = a->T;
    p.va = a->dim_a * elem / 16;
    p.vb = a->dim_b * elem / 16;
    p.ps_shift = __builtin_ctz(static_cast<unsigned>(a->page_size));
    p.all = static_cast<int64_t>(a->pages) * a->page_size;
    const hipStream_t stream = static_cast<hipStream_t>(stream_v);
    return timed_launch(sv::KK_CACHE_WRITE, stream,
                        [&](const sv::LaunchEvents& ev) { return sv::launch_cache_write(p, stream, ev); });
}

}  // namespace

extern "C" {

int spec_verify(const sv_logits* target_logits, const sv_logits* draft_logits, const int32_t* draft_tokens,
                const int32_t* draft_len, float temperature, float top_p, uint64_t seed, int32_t* out_tokens,
                int32_t* out_n_accepted, void* stream) {
    return entry([&] {
        return verify_impl(target_logits, draft_logits, draft_tokens, draft_len, temperature, top_p, seed, out_tokens,
                           out_n_accepted, nullptr, nullptr, stream);
    });
}

int spec_verify_noalloc(const sv_logits* target_logits, const sv_logits* draft_logits, const int32_t* draft_tokens,
                        const int32_t* draft_len, float temperature, float top_p, uint64_t seed, int32_t* out_tokens,
                        int32_t* out_n_accepted, void* stream) {
    return entry([&] {
        return verify_noalloc_impl(target_logits, draft_logits, draft_tokens, draft_len, temperature, top_p, seed,
                                   out_tokens, out_n_accepted, stream);
    });
}

int spec_verify_probe(const sv_logits* target_logits, const sv_logits* draft_logits, const int32_t* draft_tokens,
                      const int32_t* draft_len, float temperature, float top_p, uint64_t seed,
                      int32_t* out_tokens, int32_t* out_n_accepted, double* probe_pos, double* probe_row,
                      void* stream) {
    if (!probe_pos || !probe_row) return SV_EINVAL;
    if (misaligned(probe_pos, 8) || misaligned(probe_row, 8)) return SV_EALIGN;
    return entry([&] {
        return verify_impl(target_logits, draft_logits, draft_tokens, draft_len, temperature, top_p, seed, out_tokens,
                           out_n_accepted, probe_pos, probe_row, stream);
    });
}

int spec_greedy_verify(const sv_logits* target_logits, const int32_t* draft_tokens, const int32_t* draft_len,
                       int32_t k, int32_t* out_tokens, int32_t* out_n_accepted, int32_t* out_topk, void* stream) {
    return entry([&] {
        return greedy_impl(target_logits, draft_tokens, draft_len, k, out_tokens, out_n_accepted, out_topk, stream);
    });
}

int spec_hispec_verify(const sv_logits* final_logits, const sv_logits* inter_logits, const sv_logits* draft_logits,
                       const int32_t* draft_tokens, const int32_t* draft_len, float temperature, float top_p,
                       uint64_t seed, int32_t* out_tokens, int32_t* out_n_accepted, int32_t* out_n_stage1,
                       void* stream) {
    return entry([&] {
        return hispec_impl(final_logits, inter_logits, draft_logits, draft_tokens, draft_len, temperature, top_p, seed,
                           out_tokens, out_n_accepted, out_n_stage1, stream);
    });
}

int spec_smc_step(const sv_logits* target_logits, const sv_logits* draft_logits, const int32_t* draft_tokens,
                  const double* logw_in, float temperature, double ess_fraction, uint64_t seed, int32_t* out_bonus,
                  double* out_logw, int32_t* out_ancestor, double* out_ess, int32_t* out_resampled, void* stream) {
    return entry([&] {
        return smc_impl(target_logits, draft_logits, draft_tokens, logw_in, temperature, ess_fraction, seed, out_bonus,
                        out_logw, out_ancestor, out_ess, out_resampled, stream);
    });
}

int spec_draft_produce(const sv_logits* target_logits, int32_t K, uint64_t seed, void* draft_out,
                       int64_t out_stride_b, int64_t out_stride_p, int32_t* out_tokens, void* stream) {
    return entry([&] {
        return produce_impl(target_logits, K, seed, draft_out, out_stride_b, out_stride_p, out_tokens, stream);
    });
}

int spec_tree_attention(const sv_tree_attention* args, void* stream) {
    return entry([&] {
        return tree_attention_impl(args, stream);
    });
}

int64_t spec_tree_attention_workspace(const sv_tree_attention* args) {
    return entry([&] {
        TreePlan t;
        const int rc = plan_tree(args, t);
        return rc ? rc : static_cast<int64_t>(t.total);
    });
}

int spec_latent_attention(const sv_latent_attention* args, void* stream) {
    return entry([&] { return latent_attention_impl(args, stream); });
}

int64_t spec_latent_attention_workspace(const sv_latent_attention* args) {
    return entry([&] {
        LatentPlan t;
        const int rc = plan_latent(args, t);
        return rc ? rc : static_cast<int64_t>(t.total);
    });
}

int spec_head_product(const sv_head_product* args, void* stream) {
    return entry([&] { return head_product_impl(args, stream); });
}

int spec_latent_prompt(const sv_latent_prompt* args, void* stream) {
    return entry([&] { return latent_prompt_impl(args, stream); });
}

int64_t spec_latent_prompt_workspace(const sv_latent_prompt* args) {
    return entry([&] {
        PromptPlan t;
        const int rc = plan_prompt(args, t);
        return rc ? rc : static_cast<int64_t>(t.total);
    });
}

int spec_verify_tree(const sv_logits* target_probs, const sv_logits* draft_probs, const int32_t* tokens,
                     const int32_t* parent, const int32_t* n_nodes, const float* u_accept, const float* u_final,
                     int32_t* out_tokens, int32_t* out_nodes, int32_t* out_n_accepted, void* workspace,
                     int64_t workspace_bytes, void* stream) {
    return entry([&] {
        return verify_tree_impl(target_probs, draft_probs, tokens, parent, n_nodes, u_accept, u_final, out_tokens,
                                out_nodes, out_n_accepted, workspace, workspace_bytes, stream);
    });
}

int64_t spec_verify_tree_workspace(int32_t B, int32_t N, int32_t V, int32_t dtype, int32_t draft) {
    if (dtype != SV_F32 && dtype != SV_BF16) return SV_EDTYPE;
    if (B < 1 || B >= 1 << 22 || N < 1 || N > SPECVERIFY_MAX_NODES || V < 1 || V > SPECVERIFY_MAX_V) return SV_ESHAPE;
    return entry([&] { return verify_workspace(B, N, verify_team(B, V, dtype, draft != 0)); });
}

int spec_cache_commit(const sv_cache* cache, const void* k_tree, const void* v_tree, const int64_t k_tree_stride[4],
                      const int64_t v_tree_stride[4], int32_t N, const int32_t* nodes, const int32_t* n_accepted,
                      int32_t* out_table, int64_t out_stride, int32_t* out_len, int32_t* out_status, void* workspace,
                      int64_t workspace_bytes, void* stream) {
    return entry([&] {
        return cache_impl(cache, k_tree, v_tree, k_tree_stride, v_tree_stride, N, nodes, n_accepted, nullptr, false,
                          out_table, out_stride, out_len, out_status, workspace, workspace_bytes, stream);
    });
}

int spec_cache_fork(const sv_cache* cache, const int32_t* ancestor, int32_t* out_table, int64_t out_stride,
                    int32_t* out_len, int32_t* out_status, void* workspace, int64_t workspace_bytes, void* stream) {
    return entry([&] {
        return cache_impl(cache, nullptr, nullptr, nullptr, nullptr, 0, nullptr, nullptr, ancestor, true, out_table,
                          out_stride, out_len, out_status, workspace, workspace_bytes, stream);
    });
}

int64_t spec_cache_workspace(int32_t B, int32_t N, int32_t page_size) {
    if (B < 1 || N < 0 || !pow2_page(page_size)) return SV_ESHAPE;
    return cache_workspace(B, N, page_size);
}

int spec_beam_select(const sv_logits* logits, const float* scores, const int32_t* finished, int32_t end,
                     int32_t* out_tokens, int32_t* out_ancestor, float* out_scores, int32_t* out_finished,
                     void* workspace, int64_t workspace_bytes, void* stream) {
    return entry([&] {
        return beam_select_impl(logits, scores, finished, end, out_tokens, out_ancestor, out_scores, out_finished,
                                workspace, workspace_bytes, stream);
    });
}

int64_t spec_beam_workspace(int32_t B, int32_t W, int32_t V) {
    return entry([&] {
        const int rc = check_beams(B, W, V);
        return rc ? rc : beam_workspace(static_cast<int64_t>(B) * W, W, V);
    });
}

int spec_beam_reorder(const void* src, int64_t src_stride, void* dst, int64_t dst_stride, int64_t row_bytes,
                      int32_t rows, const int32_t* ancestor, void* stream) {
    return entry([&] {
        return beam_reorder_impl(src, src_stride, dst, dst_stride, row_bytes, rows, ancestor, stream);
    });
}

int spec_cache_reserve(const int32_t* table, int64_t table_stride, const int32_t* len, const int32_t* n_new, int32_t B,
                       int32_t width, int32_t pages, int32_t page_size, int32_t rows, int32_t* out_table,
                       int64_t out_stride, int32_t* out_len, int32_t* out_start, int32_t* out_slots,
                       int32_t* out_position, int32_t* out_status, void* workspace, int64_t workspace_bytes,
                       void* stream) {
    return entry([&] {
        return cache_reserve_impl(table, table_stride, len, n_new, B, width, pages, page_size, rows, out_table,
                                  out_stride, out_len, out_start, out_slots, out_position, out_status, workspace,
                                  workspace_bytes, stream);
    });
}

int64_t spec_cache_reserve_workspace(int32_t B, int32_t page_size, int32_t rows) {
    const int rc = check_reserve(B, page_size, rows);
    return rc ? rc : reserve_workspace(B, page_size, rows);
}

int spec_cache_write(const sv_cache_rows* args, void* stream) {
    return entry([&] { return cache_write_impl(args, stream); });
}

const char* spec_verify_strerror(int status) {
    switch (status) {
        case SV_OK: return "success";
        case SV_EINVAL: return "invalid argument (NULL pointer, temperature, top_p, scale, window or stride)";
        case SV_ESHAPE: return "invalid shape (B, K, V out of range or target/draft mismatch)";
        case SV_EDTYPE: return "invalid or mismatched dtype";
        case SV_EHIP: return g_hip_msg.empty() ? "HIP runtime error" : g_hip_msg.c_str();
        case SV_ENOMEM: return "an allocation failed";
        case SV_EALIGN: return "pointer not aligned to its element size (tree and cache rows: to 16 bytes)";
        case SV_ECAPTURE: return "the stream is being captured and the call would have to grow its scratch";
        case SV_ETOOBIG:
            return "the call needs more scratch than spec_verify_noalloc's fixed array, or the given workspace, holds";
        default: return "unknown status";
    }
}

void spec_verify_release(void) {
    std::lock_guard<std::mutex> lk(g_mu);
    for (auto& kv : g_scratch) {
        if (kv.second.ptr) (void)hipFree(kv.second.ptr);
    }
    g_scratch.clear();
    for (void* p : g_retired) (void)hipFree(p);
    g_retired.clear();
}

int spec_verify_abi_version(void) { return SPECVERIFY_ABI_VERSION; }

int spec_verify_stream_read(const void* buf, int64_t bytes, uint32_t* sink, int unroll, void* stream) {
    if (!buf || !sink || bytes < 16) return SV_EINVAL;
    if (misaligned(buf, 16) || misaligned(sink, 4)) return SV_EALIGN;
    if (unroll != 2 && unroll != 4 && unroll != 8) return SV_EINVAL;
    return entry([&] {
        const hipError_t e = sv::launch_stream_read(buf, bytes, sink, unroll, static_cast<hipStream_t>(stream));
        return e == hipSuccess ? SV_OK : hip_fail(e, "stream read launch");
    });
}

int spec_verify_profile_enable(int enable) {
    std::lock_guard<std::mutex> lk(g_mu);
    g_prof = enable != 0;
    return SV_OK;
}

int spec_verify_profile_read(double* ms, int64_t* launches, int n) {
    if (n < 0 || (n > 0 && (!ms || !launches))) return SV_EINVAL;
    return entry([&] {
        std::vector<EvPair> evs;
        {
            std::lock_guard<std::mutex> lk(g_mu);
            evs.swap(g_events);
        }
        const int kinds = n < sv::KK_ALL ? n : static_cast<int>(sv::KK_ALL);
        for (int k = 0; k < kinds; ++k) {
            ms[k] = 0.0;
            launches[k] = 0;
        }
        int rc = SV_OK;
        for (const EvPair& e : evs) {
            float t = 0.f;
            hipError_t err = hipEventSynchronize(e.b);
            if (err == hipSuccess) err = hipEventElapsedTime(&t, e.a, e.b);
            if (err != hipSuccess) rc = hip_fail(err, "hipEventElapsedTime");
            if (e.kind < kinds) {
                ms[e.kind] += t;
                launches[e.kind] += 1;
            }
            (void)hipEventDestroy(e.a);
            (void)hipEventDestroy(e.b);
        }
        return rc == SV_OK ? kinds : rc;
    });
}

}  // extern "C"
