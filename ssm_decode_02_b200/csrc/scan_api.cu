// scan_api.cu -- rsq_scan and rsq_scan_backward: validation, the workspace and the
// order of the launches.
#include <cuda_runtime.h>

#include <algorithm>

#include "tc.cuh"

namespace rsq {
namespace scan {
namespace {

constexpr int64_t kMaxTokens = (1LL << 31) - (1LL << 17);
// Longest sequences that the token-by-token kernel takes.  Its time grows with the
// tokens, that of the chunk kernels is the same for 1 and 128: 128 sequences, 80 heads
// of 128 x 64, 111, 349 and 635 us for 1, 8 and 16 tokens against 570 to 820; 4
// sequences 4.9, 15 and 27 us against 44; 16 of 16 heads of 128 x 128 6.8, 22 and 40
// against 43.
constexpr int kStepTokens = 12;
// Up to so many sequences of a ragged batch the states' blocks look for the long ones
// (long_sequence), of which there are at most tokens / 13: a block without work costs
// about 1 us of an SM, a look through 32 sequences a tenth of that.
constexpr int kLookThrough = 2048;

bool dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128 || d == 256; }
bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
// gates, their gradients and bounds are read and written one at a time
bool odd_float(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

rsq_status check_config(const char* who, const rsq_scan_config* c) {
    if (!c) return set_error(RSQ_E_INVAL, "%s: null config", who);
    if (c->family < RSQ_GDN || c->family > RSQ_KDA) return set_error(RSQ_E_INVAL, "%s: bad family %d", who, c->family);
    if (c->family != RSQ_MAMBA2)
        return set_error(RSQ_E_UNSUPPORTED, "%s: built for the scalar-decay family (RSQ_MAMBA2)", who);
    if (c->in_dtype != RSQ_F32 && c->in_dtype != RSQ_BF16) return set_error(RSQ_E_INVAL, "%s: bad in_dtype %d", who, c->in_dtype);
    if (c->in_dtype != RSQ_BF16) return set_error(RSQ_E_UNSUPPORTED, "%s: built for bf16 inputs", who);
    if (c->sequences < 1 || c->sequences > 65536) return set_error(RSQ_E_INVAL, "%s: sequences must be in [1, 65536]", who);
    if (c->heads < 1 || c->heads > RSQ_MAX_HEADS) return set_error(RSQ_E_INVAL, "%s: heads must be in [1, %d]", who, RSQ_MAX_HEADS);
    if (!dim_ok(c->dk) || !dim_ok(c->dv))
        return set_error(RSQ_E_UNSUPPORTED, "%s: dk and dv must be one of 16, 32, 64, 128, 256 (got %d, %d)", who, c->dk, c->dv);
    if (c->ngroups < 1 || c->heads % c->ngroups) return set_error(RSQ_E_INVAL, "%s: ngroups must divide heads", who);
    if (c->ragged != 0 && c->ragged != 1) return set_error(RSQ_E_INVAL, "%s: ragged must be 0 or 1", who);
    if (c->tokens < 0 || c->tokens > kMaxTokens) return set_error(RSQ_E_INVAL, "%s: tokens out of range", who);
    if (!c->ragged && c->tokens % c->sequences)
        return set_error(RSQ_E_INVAL, "%s: tokens must be a multiple of sequences (or ragged)", who);
    return RSQ_OK;
}

bool takes_steps(const rsq_scan_config& c) { return !c.ragged && c.tokens / c.sequences <= kStepTokens; }

// Sizes and the workspace's layout, offsets from `base` (null: to count bytes).
size_t layout(const rsq_scan_config& c, bool backward, Params* p, uint8_t* base) {
    p->n = c.sequences;
    p->H = c.heads;
    p->N = c.dk;
    p->P = c.dv;
    p->G = c.ngroups;
    p->per = c.heads / c.ngroups;
    p->tiles = (c.dv + kTile - 1) / kTile;
    p->ragged = c.ragged;
    p->tokens = static_cast<int>(c.tokens);
    p->len = c.ragged ? 0 : static_cast<int>(c.tokens / c.sequences);
    auto slots_of = [&](int unit) {
        if (!c.tokens) return 0;
        return c.ragged ? p->tokens / unit + p->n : p->n * ((p->len + unit - 1) / unit);
    };
    p->slots = slots_of(kChunk);
    // Segments where the sequences alone leave half of the SMs idle: twice the work on
    // the states, spread over as many blocks as run at once (a few more would take as
    // long as twice as many).
    const bool tc = states_tc_ok(*p);
    const long long blocks = static_cast<long long>(p->n) * (backward ? 2 : 1) *
                             (tc ? p->H * p->P / 128 * std::max(1, p->N / 128) : p->H * p->tiles);
    const int chunks = p->slots / p->n;
    const int fit = (tc ? 1 : 2) * kSms;
    p->seg_chunks = 0;
    if (blocks * 4 <= fit && chunks >= 16) {
        const int want = static_cast<int>(fit / blocks);
        p->seg_chunks = std::max(4, (chunks + want - 1) / want);
        if (p->seg_chunks * 2 > chunks) p->seg_chunks = 0;
    }
    p->seg_slots = p->seg_chunks ? slots_of(kChunk * p->seg_chunks) : 0;

    size_t at = 0;
    auto take = [&](size_t bytes) {
        uint8_t* q = base ? base + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return q;
    };
    const size_t cells = static_cast<size_t>(p->slots) * p->H;
    const size_t state = static_cast<size_t>(p->N) * kTile * p->tiles;
    p->flag = reinterpret_cast<unsigned*>(take(sizeof(unsigned)));
    p->rows = reinterpret_cast<int2*>(take(static_cast<size_t>(p->slots) * sizeof(int2)));
    p->gb = reinterpret_cast<float2*>(take(cells * kChunk * sizeof(float2)));
    p->gdt = reinterpret_cast<float*>(take(cells * kChunk * sizeof(float)));
    if (backward) {
        p->sf = reinterpret_cast<float*>(take(cells * state * sizeof(float)));
        p->df = reinterpret_cast<float*>(take(cells * state * sizeof(float)));
        p->part = reinterpret_cast<float*>(take(2 * cells * sizeof(float)));
    } else {
        p->sh = reinterpret_cast<bf16*>(take(cells * state * sizeof(bf16)));
    }
    if (p->seg_chunks) {
        const size_t n = static_cast<size_t>(p->seg_slots) * p->H;
        for (int d = 0; d < (backward ? 2 : 1); ++d) {
            p->seg_end[d] = reinterpret_cast<float*>(take(n * p->N * p->P * sizeof(float)));
            p->seg_start[d] = reinterpret_cast<float*>(take(n * p->N * p->P * sizeof(float)));
        }
        p->seg_log = reinterpret_cast<double*>(take(n * sizeof(double)));
    }
    return at;
}

rsq_status check_inputs(const char* who, const rsq_scan_config& c, const rsq_scan_inputs* in, const int32_t* cu, Params* p) {
    if (!in) return set_error(RSQ_E_INVAL, "%s: null inputs", who);
    const bool any = c.tokens > 0;
    if (any && (!in->x || !in->Bm || !in->Cm)) return set_error(RSQ_E_INVAL, "%s: null x, Bm or Cm", who);
    if (any && !in->decay && (!in->dt || !in->A)) return set_error(RSQ_E_INVAL, "%s: without decay, dt and A are needed", who);
    if (c.ragged && !cu) return set_error(RSQ_E_INVAL, "%s: ragged needs cu_seqlens", who);
    if (!c.ragged && cu) return set_error(RSQ_E_INVAL, "%s: cu_seqlens without ragged", who);
    for (const void* q : {in->x, in->Bm, in->Cm})
        if (misaligned(q)) return set_error(RSQ_E_INVAL, "%s: x, Bm or Cm is not 16-byte aligned", who);
    for (const void* q : {static_cast<const void*>(in->dt), static_cast<const void*>(in->A), static_cast<const void*>(in->D),
                          static_cast<const void*>(in->decay), static_cast<const void*>(cu)})
        if (odd_float(q)) return set_error(RSQ_E_INVAL, "%s: a gate array or cu_seqlens is not 4-byte aligned", who);
    const int64_t row[3] = {static_cast<int64_t>(c.heads) * c.dv, static_cast<int64_t>(c.ngroups) * c.dk,
                            static_cast<int64_t>(c.ngroups) * c.dk};
    const int64_t given[3] = {in->x_stride, in->b_stride, in->c_stride};
    long long* out[3] = {&p->xs, &p->bs, &p->cs};
    for (int i = 0; i < 3; ++i) {
        *out[i] = given[i] ? given[i] : row[i];
        if (*out[i] < row[i] || *out[i] % 8 || *out[i] > (1LL << 31))
            return set_error(RSQ_E_INVAL, "%s: a token stride must be a multiple of 8, at least the row and at most 2^31", who);
    }
    p->x = static_cast<const bf16*>(in->x);
    p->Bm = static_cast<const bf16*>(in->Bm);
    p->Cm = static_cast<const bf16*>(in->Cm);
    p->dt = in->dt;
    p->A = in->A;
    p->D = in->D;
    p->decay = in->decay;
    p->cu = cu;
    return RSQ_OK;
}

rsq_status check_workspace(const char* who, size_t need, const void* ws, size_t bytes) {
    if (!need) return RSQ_OK;
    if (!ws || misaligned(ws)) return set_error(RSQ_E_INVAL, "%s: workspace null or not 16-byte aligned", who);
    if (bytes < need) return set_error(RSQ_E_INVAL, "%s: workspace of %zu bytes, %zu needed", who, bytes, need);
    return RSQ_OK;
}

// Heads of a unit of the chunk kernels, of which an SM works on one at a time: the
// split with the fewest rounds times their length.  `start`: what the beginning of a
// unit (keys, scores) is worth in quarters of a head's tile -- two tiles where a block
// has one unit, little where the next one's beginning is hidden behind the last heads.
int head_set(const Params& p, int start) {
    // of a ragged batch about half of the sequences' last chunks come on top
    const long long chunks = std::max(1, std::min(p.slots, p.tokens / kChunk + (p.ragged ? p.n / 2 : 0)));
    int best = p.per;
    long long least = -1;
    for (int set = p.per; set >= 1; --set) {
        const long long blocks = chunks * p.G * ((p.per + set - 1) / set);
        const long long cost = (blocks + kSms - 1) / kSms * (4 * set * p.tiles + start);
        if (least < 0 || cost < least) {
            least = cost;
            best = set;
        }
    }
    return best;
}

// Launches that use none of the maps leave them out (tiles of 64 columns need dk and
// dv of 64 at least).
int maps_for(const Params& p, bool backward, tc::Maps* m) {
    return p.slots && p.N >= 64 && p.P >= 64 ? tc::make_maps(p, backward, m) : 0;
}

rsq_status done(const char* who, int err) {
    return err ? set_error(RSQ_E_CUDA, "%s: %s", who, cudaGetErrorString(static_cast<cudaError_t>(err))) : RSQ_OK;
}

}  // namespace

int tc::make_maps(const Params& p, bool backward, Maps* m) {
    // the driver's encoder, found once (the runtime library links no driver symbol)
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (!encode) return cudaErrorNotSupported;
    auto one = [&](CUtensorMap* map, const bf16* base, long long cols, long long rows, long long stride) {
        const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
        const cuuint64_t pitch[1] = {static_cast<cuuint64_t>(stride) * 2};
        const cuuint32_t box[2] = {64, 64}, step[2] = {1, 1};
        return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<bf16*>(base), dims, pitch, box, step,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    const long long hp = static_cast<long long>(p.H) * p.P, gn = static_cast<long long>(p.G) * p.N;
    bool ok = one(&m->x, p.x, hp, p.tokens, p.xs) && one(&m->Bm, p.Bm, gn, p.tokens, p.bs) && one(&m->Cm, p.Cm, gn, p.tokens, p.cs);
    if (backward)
        ok = ok && one(&m->dout, p.dout, hp, p.tokens, hp);
    else
        ok = ok && one(&m->sh, p.sh, kTile, static_cast<long long>(p.slots) * p.H * p.tiles * p.N, kTile);
    return ok ? 0 : cudaErrorInvalidValue;
}

}  // namespace scan
}  // namespace rsq

using namespace rsq;
using namespace rsq::scan;

extern "C" {

rsq_status rsq_scan_workspace(const rsq_scan_config* cfg, int backward, size_t* bytes) {
    if (!bytes) return set_error(RSQ_E_INVAL, "scan_workspace: null argument");
    const rsq_status st = check_config("scan_workspace", cfg);
    if (st) return st;
    if (backward != 0 && backward != 1) return set_error(RSQ_E_INVAL, "scan_workspace: backward must be 0 or 1");
    Params p{};
    *bytes = !backward && takes_steps(*cfg) ? 0 : layout(*cfg, backward, &p, nullptr);
    return RSQ_OK;
}

rsq_status rsq_scan(const rsq_scan_config* cfg, const rsq_scan_inputs* inputs, const int32_t* cu_seqlens,
                    const float* state_in, float* state_out, void* out, void* workspace, size_t workspace_bytes,
                    void* stream) {
    rsq_status st = check_config("scan", cfg);
    if (st) return st;
    Params p{};
    if ((st = check_inputs("scan", *cfg, inputs, cu_seqlens, &p))) return st;
    if (cfg->tokens && !out) return set_error(RSQ_E_INVAL, "scan: null out");
    if (misaligned(out) || misaligned(state_in) || misaligned(state_out))
        return set_error(RSQ_E_INVAL, "scan: out or a state is not 16-byte aligned");
    const bool steps = takes_steps(*cfg);
    if (!steps && (st = check_workspace("scan", layout(*cfg, false, &p, nullptr), workspace, workspace_bytes))) return st;
    layout(*cfg, false, &p, steps ? nullptr : static_cast<uint8_t*>(workspace));
    p.state_in = state_in;
    p.state_out = state_out;
    p.out = static_cast<bf16*>(out);
    auto s = static_cast<cudaStream_t>(stream);
    if (steps) {
        // needs no workspace, but its mark speaks of the last call with it (rsq_scan_check)
        if (workspace && !misaligned(workspace) && workspace_bytes >= sizeof(unsigned)) p.flag = static_cast<unsigned*>(workspace);
        return done("scan", launch_step(p, s));
    }
    if (cfg->ragged) {
        p.steps = kStepTokens;
        const int most = p.tokens / (kStepTokens + 1);
        if (p.n <= kLookThrough && most < p.n) p.longs = std::max(1, most);
    }
    tc::Maps m{};
    int err = maps_for(p, false, &m);
    if (!err) err = p.slots ? launch_gates(p, s) : cudaMemsetAsync(p.flag, 0, sizeof(unsigned), s);
    if (!err) err = launch_states(p, m, false, s);
    if (!err && p.steps) err = launch_step(p, s);
    if (!err && p.slots) err = launch_out(p, m, head_set(p, out_tc_ok(p) ? 1 : 8), s);
    return done("scan", err);
}

rsq_status rsq_scan_check(const void* workspace, void* stream) {
    if (!workspace || misaligned(workspace)) return set_error(RSQ_E_INVAL, "scan_check: workspace null or not 16-byte aligned");
    unsigned word = 0;   // the first of every layout
    auto s = static_cast<cudaStream_t>(stream);
    int err = cudaMemcpyAsync(&word, workspace, sizeof(word), cudaMemcpyDeviceToHost, s);
    if (!err) err = cudaStreamSynchronize(s);
    if (err) return done("scan_check", err);
    return word ? set_error(RSQ_E_CUDA, "scan_check: a bounded wait of the scan's kernels ran out") : RSQ_OK;
}

rsq_status rsq_scan_backward(const rsq_scan_config* cfg, const rsq_scan_inputs* inputs, const int32_t* cu_seqlens,
                             const float* state_in, const void* dout, const float* dstate_out,
                             const rsq_scan_grads* grads, void* workspace, size_t workspace_bytes, void* stream) {
    rsq_status st = check_config("scan_backward", cfg);
    if (st) return st;
    Params p{};
    if ((st = check_inputs("scan_backward", *cfg, inputs, cu_seqlens, &p))) return st;
    if (!grads) return set_error(RSQ_E_INVAL, "scan_backward: null grads");
    if (cfg->tokens && !dout) return set_error(RSQ_E_INVAL, "scan_backward: null dout");
    if (grads->dA && inputs->decay) return set_error(RSQ_E_INVAL, "scan_backward: dA with a given decay");
    for (const void* q : {dout, static_cast<const void*>(state_in), static_cast<const void*>(dstate_out), static_cast<const void*>(grads->dx),
                          static_cast<const void*>(grads->dBm), static_cast<const void*>(grads->dCm),
                          static_cast<const void*>(grads->dstate_in)})
        if (misaligned(q)) return set_error(RSQ_E_INVAL, "scan_backward: a buffer is not 16-byte aligned");
    for (const void* q : {static_cast<const void*>(grads->ddt), static_cast<const void*>(grads->dlog_decay),
                          static_cast<const void*>(grads->dA), static_cast<const void*>(grads->dD)})
        if (odd_float(q)) return set_error(RSQ_E_INVAL, "scan_backward: a gate gradient is not 4-byte aligned");
    if ((st = check_workspace("scan_backward", layout(*cfg, true, &p, nullptr), workspace, workspace_bytes))) return st;
    layout(*cfg, true, &p, static_cast<uint8_t*>(workspace));
    p.state_in = state_in;
    p.dout = static_cast<const bf16*>(dout);
    p.dstate_out = dstate_out;
    p.dx = static_cast<bf16*>(grads->dx);
    p.dBm = static_cast<bf16*>(grads->dBm);
    p.dCm = static_cast<bf16*>(grads->dCm);
    p.ddt = grads->ddt;
    p.dlog = grads->dlog_decay;
    p.dA = grads->dA;
    p.dD = grads->dD;
    p.dstate_in = grads->dstate_in;
    auto s = static_cast<cudaStream_t>(stream);
    tc::Maps m{};
    int err = maps_for(p, true, &m);
    if (!err) err = p.slots ? launch_gates(p, s) : cudaMemsetAsync(p.flag, 0, sizeof(unsigned), s);
    if (!err) err = launch_states(p, m, true, s);
    if (!err) err = launch_backward(p, m, head_set(p, 8), s);
    return done("scan_backward", err);
}

}  // extern "C"
