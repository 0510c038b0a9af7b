// C ABI of epx (declared in include/epx.h): host-side validation, sizing and
// kernel launches.  No call allocates, frees or synchronizes; every kernel
// goes onto the caller's stream.
#include <math.h>
#include <string.h>

#include <mutex>

#include <algorithm>

#include "epx_device.h"

// Built-in workspace of ep_dispatch_layout_noalloc, for callers that cannot
// allocate: zero when the code object loads, and each GPU the library runs
// on holds its own copy for the life of the process.  On the host the name
// is only a stand-in for the device array; host code uses the address
// scratch_address() looks up, never the name.
static __device__ __align__(256) uint8_t scratch[EP_NOALLOC_SCRATCH_BYTES];

namespace {

using namespace epx;

struct Shape {
    int32_t T, H, E, S, K, Kp, A, C, shared, src, E_loc, G, NG;
    int64_t R, min_rows, ws_bytes, tiles, chunks, sp_tiles;
    uint32_t flags;
};

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// A buffer of `bytes` bytes must be present and aligned unless it is empty.
bool bad_buffer(const void* p, int64_t bytes, uintptr_t align) {
    if (bytes == 0) return false;
    return p == nullptr || misaligned(p, align);
}

// Validate `c` and derive the sizes every call needs.
int derive(const ep_cfg_t* c, Shape* d) {
    if (c == nullptr) return EP_EINVAL;
    if (c->num_tokens < 0 || c->hidden < 8 || c->hidden % 8 != 0) return EP_EINVAL;
    if (c->num_experts < 1 || c->num_segments < 1 || c->num_experts % c->num_segments != 0) return EP_EINVAL;
    if (c->top_k < 1 || c->top_k > c->num_experts) return EP_EINVAL;
    if (c->align < 1 || c->align > (1 << 30) || c->seg_capacity < 0) return EP_EINVAL;
    if (c->shared_expert != 0 && c->shared_expert != 1) return EP_EINVAL;
    if (c->shared_expert && (c->src_segment < 0 || c->src_segment >= c->num_segments)) return EP_EINVAL;
    if (c->reserved0 != 0 || c->reserved1 != 0) return EP_EINVAL;
    constexpr uint32_t kPaths = EP_LAYOUT_LOOKBACK | EP_LAYOUT_DIRECT | EP_LAYOUT_BARRIER | EP_LAYOUT_COUNT;
    if (c->flags & ~(EP_ZERO_PAD_ROWS | kPaths)) return EP_EINVAL;
    if (__builtin_popcount(c->flags & kPaths) > 1) return EP_EINVAL;  // at most one path
    if ((c->flags & EP_LAYOUT_COUNT) && (int64_t)c->num_tokens * c->top_k > kCountForcedMaxSlots) return EP_EINVAL;
    if ((c->flags & EP_LAYOUT_BARRIER) && (int64_t)c->num_tokens * c->top_k > kBarrierForcedMaxSlots) return EP_EINVAL;
    d->T = c->num_tokens;
    d->H = c->hidden;
    d->E = c->num_experts;
    d->S = c->num_segments;
    d->K = c->top_k;
    d->shared = c->shared_expert;
    d->Kp = d->K + d->shared;
    if (d->Kp > kMaxSlots) return EP_EINVAL;  // a token's slots are spread over one wave's lanes
    d->A = c->align;
    d->C = c->seg_capacity;
    d->src = d->shared ? c->src_segment : 0;
    d->E_loc = d->E / d->S;
    d->G = d->E_loc + d->shared;
    const int64_t ng = (int64_t)d->S * d->G;
    if (ng > EP_MAX_GROUPS) return EP_EINVAL;
    d->NG = (int32_t)ng;
    const int64_t slots = (int64_t)d->T * d->Kp;
    if (slots >= (int64_t(1) << 30)) return EP_EINVAL;  // look-back descriptors hold 30-bit counts
    // Every group is padded by at most A - 1 rows, so the used rows of all
    // segments before any capacity clamp are at most `packed`.  The layout
    // kernels add up the aligned group sizes in int32 before clamping them to
    // C, so this bound must fit in int32 in capacity mode too.
    const int64_t groups = (int64_t)d->E + d->shared;
    const int64_t packed = slots + (slots < groups ? slots : groups) * (int64_t)(d->A - 1);
    if (packed >= (int64_t(1) << 31)) return EP_EINVAL;
    d->min_rows = d->C > 0 ? (int64_t)d->S * d->C : packed;
    if (d->min_rows >= (int64_t(1) << 31)) return EP_EINVAL;  // rows are int32
    // Workspace: a header, then either path's tables (the direct path's
    // 32-bit tile counts and chunk sums; the single pass's two arrays of
    // 64-bit descriptors).
    d->tiles = layout_tiles((int64_t)d->T * d->K, d->NG);
    d->chunks = direct_chunks(d->tiles);
    d->sp_tiles = sp_tiles((int64_t)d->T * d->K);
    d->ws_bytes = kWorkspaceHeader + std::max((d->tiles + d->chunks) * (int64_t)d->NG * 4,
                                              d->sp_tiles * (int64_t)d->NG * 16);
    d->R = c->recv_rows;
    d->flags = c->flags;
    return EP_OK;
}

int check_rows(const Shape& d) {
    if (d.R < d.min_rows || d.R >= (int64_t(1) << 31)) return EP_EINVAL;
    return EP_OK;
}

// The current device must be a gfx950; the answer is cached per device.
int check_device() {
    static std::mutex mu;
    static int arch_state[64];  // 0 unknown, 1 ok, 2 not supported
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return EP_ELAUNCH;
    if (dev < 0 || dev >= 64) return EP_ENOTSUP;
    std::lock_guard<std::mutex> lock(mu);
    if (arch_state[dev] == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return EP_ELAUNCH;
        arch_state[dev] = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
    }
    return arch_state[dev] == 1 ? EP_OK : EP_ENOTSUP;
}

int status_of(hipError_t e) { return e == hipSuccess ? EP_OK : EP_ELAUNCH; }

// Kernels that launch one grid for the whole batch, with `per_token`
// work-items per token: a grid dimension holds at most 2^32 - 1 work-items
// (the movers split larger batches into chunks instead).
bool grid_too_big(const Shape& d, int64_t per_token) {
    return (int64_t)d.T * per_token + 1024 > 0xFFFFFFFFll;
}

// Layout arrays read by the payload calls.
int check_layout_for_payload(const Shape& d, const ep_layout_t* L) {
    if (L == nullptr) return EP_EINVAL;
    if (bad_buffer(L->token_row, (int64_t)d.T * d.Kp * 4, 4)) return EP_EINVAL;
    if (d.flags & EP_ZERO_PAD_ROWS) {
        if (bad_buffer(L->counts, (int64_t)d.NG * 4, 4) ||
            bad_buffer(L->row_offsets, (int64_t)d.S * (d.G + 1) * 4, 4) ||
            bad_buffer(L->seg_base, (int64_t)(d.S + 1) * 4, 4))
            return EP_EINVAL;
    }
    return EP_OK;
}

MoveArgs move_args(const Shape& d, const ep_layout_t* L, const void* src, void* dst, const float* probs) {
    MoveArgs m;
    m.src = src;
    m.dst = dst;
    m.token_row = L->token_row;
    m.probs = probs;
    m.T = d.T;
    m.K = d.K;
    m.Kp = d.Kp;
    m.H = d.H;
    m.R = d.R;
    return m;
}

int zero_pad(const Shape& d, const ep_layout_t* L, void* base, int64_t row_bytes, hipStream_t st) {
    if (!(d.flags & EP_ZERO_PAD_ROWS) || d.A == 1) return EP_OK;
    return status_of(launch_zero_pad_rows(base, row_bytes, *L, d.S, d.G, d.A, d.C, d.R, st));
}

Nvfp4Args nvfp4_args(const Shape& d, const ep_layout_t* L, const uint16_t* x, uint8_t* codes, uint8_t* scales,
                     uint16_t* rowscale) {
    Nvfp4Args a;
    a.x = x;
    a.codes = codes;
    a.scales = scales;
    a.rowscale = rowscale;
    a.token_row = L->token_row;
    a.T = d.T;
    a.Kp = d.Kp;
    a.H = d.H;
    a.R = d.R;
    return a;
}

Fp8Args fp8_args(const Shape& d, const ep_layout_t* L, const uint16_t* x, uint8_t* codes, float* scales) {
    Fp8Args a;
    a.x = x;
    a.codes = codes;
    a.scales = scales;
    a.token_row = L->token_row;
    a.T = d.T;
    a.Kp = d.Kp;
    a.H = d.H;
    a.R = d.R;
    return a;
}

int zero_pad_fp8(const Shape& d, const ep_layout_t* L, uint8_t* codes, float* scales, hipStream_t st) {
    int rc;
    if ((rc = zero_pad(d, L, codes, d.H, st)) != EP_OK) return rc;
    return zero_pad(d, L, scales, (int64_t)(d.H / 128) * 4, st);
}

int zero_pad_nvfp4(const Shape& d, const ep_layout_t* L, uint8_t* codes, uint8_t* scales, uint16_t* rowscale,
                   hipStream_t st) {
    int rc;
    if ((rc = zero_pad(d, L, codes, d.H / 2, st)) != EP_OK) return rc;
    if ((rc = zero_pad(d, L, scales, d.H / 16, st)) != EP_OK) return rc;
    return zero_pad(d, L, rowscale, 2, st);
}

// Host-side checks shared by both layout entry points (everything but the
// workspace).
int layout_check(const Shape& d, const int32_t* topk_ids, const ep_layout_t* L) {
    int rc;
    if ((rc = check_rows(d)) != EP_OK) return rc;
    if ((int64_t)d.T * d.K > kLayoutMaxSlots) return EP_EINVAL;
    if (L == nullptr) return EP_EINVAL;
    if (bad_buffer(topk_ids, (int64_t)d.T * d.K * 4, 4)) return EP_EINVAL;
    if (bad_buffer(L->counts, (int64_t)d.NG * 4, 4) || bad_buffer(L->seg_base, (int64_t)(d.S + 1) * 4, 4) ||
        bad_buffer(L->row_offsets, (int64_t)d.S * (d.G + 1) * 4, 4) ||
        bad_buffer(L->scales_offsets, (int64_t)d.S * (d.G + 1) * 4, 4) ||
        bad_buffer(L->token_row, (int64_t)d.T * d.Kp * 4, 4) || bad_buffer(L->expert_ids, d.R * 4, 4) ||
        bad_buffer(L->src_info, d.R * 8, 8) || bad_buffer(L->flags, 4, 4))
        return EP_EINVAL;
    return EP_OK;
}

// Launch of the layout kernels, after layout_check and check_device; `ws`
// holds at least d.ws_bytes bytes.  With x and one dispatch's outputs given
// (out), the small path also makes that bf16, NVFP4 or FP8 dispatch
// (*fused is set when it did).
struct FusedOut {  // the dispatch a small-path layout launch makes beside the layout
    uint16_t* recv = nullptr;
    uint8_t* codes = nullptr;
    uint8_t* scales = nullptr;
    uint16_t* rowscale = nullptr;
    uint8_t* f8_codes = nullptr;
    float* f8_scales = nullptr;
};

int layout_launch(const Shape& d, const int32_t* topk_ids, void* ws, const ep_layout_t* L, void* stream,
                  const uint16_t* x = nullptr, const FusedOut& out = FusedOut(), bool* fused = nullptr) {
    LayoutArgs a;
    a.x = nullptr;
    a.recv = nullptr;
    a.codes = nullptr;
    a.scales = nullptr;
    a.rowscale = nullptr;
    a.f8_codes = nullptr;
    a.f8_scales = nullptr;
    a.fused_rpu = 1;
    a.H = d.H;
    a.topk_ids = topk_ids;
    a.desc = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + kWorkspaceHeader);
    a.out = *L;
    a.T = d.T;
    a.K = d.K;
    a.Kp = d.Kp;
    a.E = d.E;
    a.S = d.S;
    a.G = d.G;
    a.NG = d.NG;
    a.E_loc = d.E_loc;
    a.A = d.A;
    a.C = d.C;
    a.shared = d.shared;
    a.src_seg = d.src;
    a.recv_rows = d.R;
    a.sp_header = ws;
    a.sp_desc = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(ws) + kWorkspaceHeader);
    const int64_t routed = (int64_t)d.T * d.K;
    a.lookback = 0;
    if (d.flags & EP_LAYOUT_LOOKBACK) {
        a.mode = kLayoutSinglePass;
        a.lookback = 1;
    } else if (d.flags & EP_LAYOUT_BARRIER) {
        a.mode = kLayoutSinglePass;
    } else if (d.flags & EP_LAYOUT_DIRECT) {
        a.mode = kLayoutDirect;
    } else if (d.flags & EP_LAYOUT_COUNT) {
        a.mode = kLayoutCount;
    } else if (routed <= kSmallMaxSlots) {
        a.mode = kLayoutSmall;
    } else if (routed <= kCountMaxSlots) {
        a.mode = kLayoutCount;
    } else {
        a.mode = kLayoutDirect;  // measured faster than the single pass at every size
    }
    a.chunks = 0;
    a.chunk_sums = nullptr;
    if (a.mode == kLayoutSinglePass) {
        a.tiles = (int32_t)d.sp_tiles;
        a.rank_blocks = (int32_t)sp_blocks(d.sp_tiles, d.NG);
        a.slots_per_thread = sp_slots_per_thread(routed);
    } else if (a.mode == kLayoutCount) {
        a.slots_per_thread = 1;
        a.tiles = (int32_t)std::max<int64_t>(1, (routed + kLayoutThreads - 1) / kLayoutThreads);
        a.rank_blocks = (int32_t)std::max<int64_t>(a.tiles, std::min<int32_t>(d.NG, 256));
    } else if (a.mode == kLayoutDirect) {
        a.tiles = (int32_t)d.tiles;
        a.chunks = (int32_t)d.chunks;
        if (d.chunks > 0) a.chunk_sums = a.desc + d.tiles * (int64_t)d.NG;
        a.rank_blocks = (int32_t)std::max<int64_t>(d.tiles, std::min<int32_t>(d.NG, 256));
        a.slots_per_thread = layout_slots_per_thread(routed, d.NG);
    } else {  // one tile holds every slot
        a.tiles = 1;
        a.rank_blocks = std::min<int32_t>(d.NG, 256);
        a.slots_per_thread = routed <= 256 ? 1 : (routed <= 512 ? 2 : 4);
        a.x = x;
        a.recv = out.recv;
        a.codes = out.codes;
        a.scales = out.scales;
        a.rowscale = out.rowscale;
        a.f8_codes = out.f8_codes;
        a.f8_scales = out.f8_scales;
        if (x != nullptr) {
            // A fused dispatch unit is a token and up to rpu of its K' rows:
            // the fewest rows per unit whose units fit one round of
            // workgroups, so that as many tokens as possible are read (and
            // quantized) once per unit and no workgroup takes two units.
            // Measured at DeepSeek-V3 dims, T = 40 and 64: NVFP4 7.8 and 7.9
            // us against 9.0 and 9.1 with one token (all rows) per unit.
            const int64_t items = (int64_t)d.T * d.Kp, grid = a.rank_blocks;
            int32_t r = (int32_t)std::min<int64_t>(d.Kp, std::max<int64_t>(1, (items + grid - 1) / grid));
            while (r < d.Kp && (int64_t)d.T * ((d.Kp + r - 1) / r) > grid) ++r;
            a.fused_rpu = r;
        }
    }
    if (fused) *fused = a.x != nullptr;
    return status_of(launch_layout(a, static_cast<hipStream_t>(stream)));
}

// ep_route_t against the configuration.
int check_route(const Shape& d, const ep_route_t* r) {
    if (r == nullptr) return EP_EINVAL;
    if (r->score != EP_SCORE_SOFTMAX && r->score != EP_SCORE_SIGMOID) return EP_EINVAL;
    if (r->normalize != 0 && r->normalize != 1) return EP_EINVAL;
    if (r->num_groups < 1 || r->num_groups > EP_MAX_ROUTE_GROUPS || d.E % r->num_groups != 0) return EP_EINVAL;
    if (r->top_groups < 1 || r->top_groups > r->num_groups) return EP_EINVAL;
    if (!isfinite(r->scale)) return EP_EINVAL;
    if (r->logits_type != EP_TYPE_F32 && r->logits_type != EP_TYPE_BF16) return EP_EINVAL;
    if (r->reserved0 != 0 || r->reserved1 != 0) return EP_EINVAL;
    if (d.E > EP_MAX_GROUPS) return EP_EINVAL;
    return EP_OK;
}

TopkArgs topk_args(const Shape& d, const ep_route_t* r, const void* logits) {
    TopkArgs a = {};
    a.logits = logits;
    a.T = d.T;
    a.E = d.E;
    a.K = d.K;
    a.sigmoid = r->score == EP_SCORE_SIGMOID;
    a.normalize = r->normalize;
    a.groups = r->num_groups;
    a.top_groups = r->top_groups;
    a.bf16 = r->logits_type == EP_TYPE_BF16;
    a.scale = r->scale;
    return a;
}

// The experts' products: the layout arrays they read, and their dimensions.
int check_expert(const Shape& d, const ep_layout_t* L, int32_t in_dim, int32_t out_dim, int32_t in_multiple) {
    int rc;
    if ((rc = check_rows(d)) != EP_OK) return rc;
    if (in_dim < in_multiple || in_dim > EP_MAX_EXPERT_DIM || in_dim % in_multiple != 0) return EP_EINVAL;
    if (out_dim < 8 || out_dim > EP_MAX_EXPERT_DIM || out_dim % 8 != 0) return EP_EINVAL;
    if (L == nullptr || bad_buffer(L->counts, (int64_t)d.NG * 4, 4) ||
        bad_buffer(L->row_offsets, (int64_t)d.S * (d.G + 1) * 4, 4) ||
        bad_buffer(L->seg_base, (int64_t)(d.S + 1) * 4, 4))
        return EP_EINVAL;
    return EP_OK;
}

// A product whose tiles pass one grid is an argument error, found before the launch.
int expert_status(hipError_t e) { return e == hipErrorInvalidConfiguration ? EP_EINVAL : status_of(e); }

ExpertArgs expert_args(const Shape& d, const ep_layout_t* L, int32_t in_dim, int32_t out_dim, void* out) {
    ExpertArgs a = {};
    a.out = out;
    a.counts = L->counts;
    a.seg_base = L->seg_base;
    a.row_offsets = L->row_offsets;
    a.in = in_dim;
    a.on = out_dim;
    a.E = d.E;
    a.S = d.S;
    a.G = d.G;
    a.NG = d.NG;
    a.E_loc = d.E_loc;
    a.C = d.C;
    a.shared = d.shared;
    a.src_seg = d.src;
    a.R = d.R;
    a.slots = std::min<int64_t>((int64_t)d.T * d.Kp, d.R);
    return a;
}

// Adapters against the configuration; a and b as the call reads them.
int check_lora(const Shape& d, const ep_lora_t* l, bool reads_a, bool reads_b) {
    if (l == nullptr || l->reserved0 != 0 || l->reserved1 != 0) return EP_EINVAL;
    if (l->num_adapters < 1 || l->num_adapters > EP_MAX_ADAPTERS) return EP_EINVAL;
    if (l->rank < 8 || l->rank > EP_MAX_LORA_RANK || l->rank % 8 != 0) return EP_EINVAL;
    if (bad_buffer(l->token_adapter, (int64_t)d.T * 4, 4) || misaligned(l->scale, 4)) return EP_EINVAL;
    if ((reads_a && bad_buffer(l->a, 16, 16)) || (reads_b && bad_buffer(l->b, 16, 16))) return EP_EINVAL;
    return EP_OK;
}

// What the gated block and the calls with adapters read of the layout.
int check_block(const Shape& d, const ep_layout_t* L, int32_t in_dim, int32_t out_dim, int32_t in_multiple) {
    const int rc = check_expert(d, L, in_dim, out_dim, in_multiple);
    if (rc != EP_OK) return rc;
    return bad_buffer(L->src_info, d.R * 8, 8) ? EP_EINVAL : EP_OK;
}

BlockArgs block_args(const Shape& d, const ep_layout_t* L, const ep_lora_t* l, int32_t in_dim, int32_t out_dim,
                     const float* u, void* out) {
    BlockArgs a = {};
    a.e = expert_args(d, L, in_dim, out_dim, out);
    if (l != nullptr) a.l = {l->token_adapter, l->a, l->b, l->scale, l->num_adapters, l->rank};
    a.u = u;
    a.src_info = L->src_info;
    a.token_row = L->token_row;
    a.T = d.T;
    a.K = d.K;
    a.Kp = d.Kp;
    return a;
}

// Of the gated block: inter columns of act, optional adapters.
int check_gated(const Shape& d, const ep_layout_t* L, const ep_lora_t* l, int32_t in_dim, int32_t inter,
                int32_t in_multiple, const float* ulora, const float* probs) {
    int rc;
    if ((rc = check_block(d, L, in_dim, inter, in_multiple)) != EP_OK) return rc;
    if (l != nullptr) {
        if ((rc = check_lora(d, l, false, true)) != EP_OK) return rc;
        if (bad_buffer(ulora, d.R * l->rank * 4, 16)) return EP_EINVAL;
    } else if (ulora != nullptr) {
        return EP_EINVAL;
    }
    return misaligned(probs, 4) ? EP_EINVAL : EP_OK;
}

BlockArgs gated_args(const Shape& d, const ep_layout_t* L, const ep_lora_t* l, int32_t in_dim, int32_t inter,
                     const float* ulora, const float* probs, void* act) {
    BlockArgs a = block_args(d, L, l, in_dim, 2 * inter, ulora, act);
    a.probs = probs;
    a.I = inter;
    return a;
}

constexpr int64_t kScratchBytes = EP_NOALLOC_SCRATCH_BYTES;

// Device address of `scratch` on the current device, looked up once per
// device (with that device current) and kept.
int scratch_address(void** out) {
    static std::mutex mu;
    static void* addr[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return EP_ELAUNCH;
    if (dev < 0 || dev >= 64) return EP_ENOTSUP;
    std::lock_guard<std::mutex> lock(mu);
    if (addr[dev] == nullptr) {
        void* p = nullptr;
        if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || p == nullptr) return EP_ELAUNCH;
        addr[dev] = p;
    }
    *out = addr[dev];
    return EP_OK;
}

}  // namespace

extern "C" {

int ep_abi_version(void) { return EPX_ABI_VERSION; }

const char* ep_strerror(int status) {
    switch (status) {
        case EP_OK: return "ok";
        case EP_EINVAL: return "invalid argument";
        case EP_ELAUNCH: return "HIP runtime error while enqueueing work";
        case EP_ENOTSUP: return "device is not gfx950 (MI355X)";
        case EP_ESCRATCH:
            return "the layout needs more scratch than the built-in buffer of ep_dispatch_layout_noalloc "
                   "holds (EP_NOALLOC_SCRATCH_BYTES); use ep_dispatch_layout with a workspace";
        default: return "unknown status";
    }
}

int ep_query(const ep_cfg_t* cfg, int64_t* min_recv_rows, int64_t* workspace_bytes, int32_t* groups_per_seg) {
    Shape d;
    const int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if (min_recv_rows) *min_recv_rows = d.min_rows;
    if (workspace_bytes) *workspace_bytes = d.ws_bytes;
    if (groups_per_seg) *groups_per_seg = d.G;
    return EP_OK;
}

int ep_dispatch_layout(const ep_cfg_t* cfg, const int32_t* topk_ids, void* workspace, int64_t workspace_bytes,
                       const ep_layout_t* layout, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = layout_check(d, topk_ids, layout)) != EP_OK) return rc;
    if (workspace == nullptr || misaligned(workspace, 16) || workspace_bytes < d.ws_bytes) return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    return layout_launch(d, topk_ids, workspace, layout, stream);
}

int ep_dispatch_layout_noalloc(const ep_cfg_t* cfg, const int32_t* topk_ids, const ep_layout_t* layout,
                               void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = layout_check(d, topk_ids, layout)) != EP_OK) return rc;
    if (d.ws_bytes > kScratchBytes) return EP_ESCRATCH;
    if ((rc = check_device()) != EP_OK) return rc;
    void* ws = nullptr;
    if ((rc = scratch_address(&ws)) != EP_OK) return rc;
    return layout_launch(d, topk_ids, ws, layout, stream);
}

int ep_dispatch(const ep_cfg_t* cfg, const ep_layout_t* layout, const uint16_t* x, uint16_t* recv, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_rows(d)) != EP_OK) return rc;
    if ((rc = check_layout_for_payload(d, layout)) != EP_OK) return rc;
    if (bad_buffer(x, (int64_t)d.T * d.H * 2, 16) || bad_buffer(recv, d.R * d.H * 2, 16)) return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if ((rc = status_of(launch_scatter(move_args(d, layout, x, recv, nullptr), st))) != EP_OK) return rc;
    return zero_pad(d, layout, recv, (int64_t)d.H * 2, st);
}

int ep_dispatch_with_layout(const ep_cfg_t* cfg, const int32_t* topk_ids, void* workspace, int64_t workspace_bytes,
                            const ep_layout_t* layout, const uint16_t* x, uint16_t* recv, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = layout_check(d, topk_ids, layout)) != EP_OK) return rc;
    if (workspace == nullptr || misaligned(workspace, 16) || workspace_bytes < d.ws_bytes) return EP_EINVAL;
    if (bad_buffer(x, (int64_t)d.T * d.H * 2, 16) || bad_buffer(recv, d.R * d.H * 2, 16)) return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    bool fused = false;
    FusedOut out;
    out.recv = recv;
    if ((rc = layout_launch(d, topk_ids, workspace, layout, stream, x, out, &fused)) != EP_OK) return rc;
    if (!fused && (rc = status_of(launch_scatter(move_args(d, layout, x, recv, nullptr), st))) != EP_OK) return rc;
    return zero_pad(d, layout, recv, (int64_t)d.H * 2, st);
}

int ep_dispatch_nvfp4(const ep_cfg_t* cfg, const ep_layout_t* layout, const uint16_t* x, uint8_t* codes,
                      uint8_t* scales, uint16_t* rowscale, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_rows(d)) != EP_OK) return rc;
    if (d.H % 16 != 0 || d.H > nvfp4_max_hidden() || grid_too_big(d, 64)) return EP_EINVAL;
    if ((rc = check_layout_for_payload(d, layout)) != EP_OK) return rc;
    if (bad_buffer(x, (int64_t)d.T * d.H * 2, 16) || bad_buffer(codes, d.R * (d.H / 2), 16) ||
        bad_buffer(scales, d.R * (d.H / 16), 1) || bad_buffer(rowscale, d.R * 2, 2))
        return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if ((rc = status_of(launch_nvfp4(nvfp4_args(d, layout, x, codes, scales, rowscale), st))) != EP_OK) return rc;
    return zero_pad_nvfp4(d, layout, codes, scales, rowscale, st);
}

int ep_dispatch_nvfp4_with_layout(const ep_cfg_t* cfg, const int32_t* topk_ids, void* workspace,
                                  int64_t workspace_bytes, const ep_layout_t* layout, const uint16_t* x,
                                  uint8_t* codes, uint8_t* scales, uint16_t* rowscale, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = layout_check(d, topk_ids, layout)) != EP_OK) return rc;
    if (workspace == nullptr || misaligned(workspace, 16) || workspace_bytes < d.ws_bytes) return EP_EINVAL;
    if (d.H % 16 != 0 || d.H > nvfp4_max_hidden() || grid_too_big(d, 64)) return EP_EINVAL;
    if (bad_buffer(x, (int64_t)d.T * d.H * 2, 16) || bad_buffer(codes, d.R * (d.H / 2), 16) ||
        bad_buffer(scales, d.R * (d.H / 16), 1) || bad_buffer(rowscale, d.R * 2, 2))
        return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    bool fused = false;
    FusedOut out;
    out.codes = codes;
    out.scales = scales;
    out.rowscale = rowscale;
    if ((rc = layout_launch(d, topk_ids, workspace, layout, stream, x, out, &fused)) != EP_OK) return rc;
    if (!fused && (rc = status_of(launch_nvfp4(nvfp4_args(d, layout, x, codes, scales, rowscale), st))) != EP_OK)
        return rc;
    return zero_pad_nvfp4(d, layout, codes, scales, rowscale, st);
}

int ep_dispatch_fp8(const ep_cfg_t* cfg, const ep_layout_t* layout, const uint16_t* x, uint8_t* codes,
                    float* scales, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_rows(d)) != EP_OK) return rc;
    if (d.H % 128 != 0 || d.H > fp8_max_hidden() || grid_too_big(d, 64)) return EP_EINVAL;
    if ((rc = check_layout_for_payload(d, layout)) != EP_OK) return rc;
    if (bad_buffer(x, (int64_t)d.T * d.H * 2, 16) || bad_buffer(codes, d.R * d.H, 16) ||
        bad_buffer(scales, d.R * (d.H / 128) * 4, 4))
        return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if ((rc = status_of(launch_fp8(fp8_args(d, layout, x, codes, scales), st))) != EP_OK) return rc;
    return zero_pad_fp8(d, layout, codes, scales, st);
}

int ep_dispatch_fp8_with_layout(const ep_cfg_t* cfg, const int32_t* topk_ids, void* workspace,
                                int64_t workspace_bytes, const ep_layout_t* layout, const uint16_t* x,
                                uint8_t* codes, float* scales, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = layout_check(d, topk_ids, layout)) != EP_OK) return rc;
    if (workspace == nullptr || misaligned(workspace, 16) || workspace_bytes < d.ws_bytes) return EP_EINVAL;
    if (d.H % 128 != 0 || d.H > fp8_max_hidden() || grid_too_big(d, 64)) return EP_EINVAL;
    if (bad_buffer(x, (int64_t)d.T * d.H * 2, 16) || bad_buffer(codes, d.R * d.H, 16) ||
        bad_buffer(scales, d.R * (d.H / 128) * 4, 4))
        return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    bool fused = false;
    FusedOut out;
    out.f8_codes = codes;
    out.f8_scales = scales;
    if ((rc = layout_launch(d, topk_ids, workspace, layout, stream, x, out, &fused)) != EP_OK) return rc;
    if (!fused && (rc = status_of(launch_fp8(fp8_args(d, layout, x, codes, scales), st))) != EP_OK) return rc;
    return zero_pad_fp8(d, layout, codes, scales, st);
}

int ep_combine(const ep_cfg_t* cfg, const ep_layout_t* layout, const uint16_t* expert_out, const float* probs,
               uint16_t* y, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_rows(d)) != EP_OK) return rc;
    if (layout == nullptr || bad_buffer(layout->token_row, (int64_t)d.T * d.Kp * 4, 4)) return EP_EINVAL;
    if (bad_buffer(expert_out, d.R * d.H * 2, 16) || bad_buffer(y, (int64_t)d.T * d.H * 2, 16)) return EP_EINVAL;
    if (probs != nullptr && misaligned(probs, 4)) return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    return status_of(launch_gather_reduce(move_args(d, layout, expert_out, y, probs), static_cast<hipStream_t>(stream)));
}

int ep_combine_nvfp4(const ep_cfg_t* cfg, const ep_layout_t* layout, const uint8_t* codes, const uint8_t* scales,
                     const uint16_t* rowscale, const float* probs, uint16_t* y, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_rows(d)) != EP_OK) return rc;
    if (d.H % 16 != 0 || grid_too_big(d, (int64_t)kWave * combine_nvfp4_pieces(d.H))) return EP_EINVAL;
    if (layout == nullptr || bad_buffer(layout->token_row, (int64_t)d.T * d.Kp * 4, 4)) return EP_EINVAL;
    if (bad_buffer(codes, d.R * (d.H / 2), 8) || bad_buffer(scales, d.R * (d.H / 16), 1) ||
        bad_buffer(rowscale, d.R * 2, 2) || bad_buffer(y, (int64_t)d.T * d.H * 2, 16))
        return EP_EINVAL;
    if (probs != nullptr && misaligned(probs, 4)) return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    CombineNvfp4Args a;
    a.codes = codes;
    a.scales = scales;
    a.rowscale = rowscale;
    a.token_row = layout->token_row;
    a.probs = probs;
    a.y = y;
    a.T = d.T;
    a.K = d.K;
    a.Kp = d.Kp;
    a.H = d.H;
    a.R = d.R;
    return status_of(launch_combine_nvfp4(a, static_cast<hipStream_t>(stream)));
}

int ep_dispatch_bwd(const ep_cfg_t* cfg, const ep_layout_t* layout, const uint16_t* grad_recv, uint16_t* grad_x,
                    void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_rows(d)) != EP_OK) return rc;
    if (layout == nullptr || bad_buffer(layout->token_row, (int64_t)d.T * d.Kp * 4, 4)) return EP_EINVAL;
    if (bad_buffer(grad_recv, d.R * d.H * 2, 16) || bad_buffer(grad_x, (int64_t)d.T * d.H * 2, 16)) return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    return status_of(launch_gather_reduce(move_args(d, layout, grad_recv, grad_x, nullptr), static_cast<hipStream_t>(stream)));
}

int ep_combine_bwd(const ep_cfg_t* cfg, const ep_layout_t* layout, const uint16_t* grad_y, const float* probs,
                   uint16_t* grad_expert_out, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_rows(d)) != EP_OK) return rc;
    if ((rc = check_layout_for_payload(d, layout)) != EP_OK) return rc;
    if (bad_buffer(grad_y, (int64_t)d.T * d.H * 2, 16) || bad_buffer(grad_expert_out, d.R * d.H * 2, 16))
        return EP_EINVAL;
    if (probs != nullptr && misaligned(probs, 4)) return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const MoveArgs m = move_args(d, layout, grad_y, grad_expert_out, probs);
    rc = status_of(probs != nullptr ? launch_scatter_scaled(m, st) : launch_scatter(m, st));
    if (rc != EP_OK) return rc;
    return zero_pad(d, layout, grad_expert_out, (int64_t)d.H * 2, st);
}

int ep_combine_bwd_probs(const ep_cfg_t* cfg, const ep_layout_t* layout, const uint16_t* grad_y,
                         const uint16_t* expert_out, float* grad_probs, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_rows(d)) != EP_OK) return rc;
    if (layout == nullptr || bad_buffer(layout->token_row, (int64_t)d.T * d.Kp * 4, 4)) return EP_EINVAL;
    if (grid_too_big(d, 256)) return EP_EINVAL;
    if (bad_buffer(grad_y, (int64_t)d.T * d.H * 2, 16) || bad_buffer(expert_out, d.R * d.H * 2, 16) ||
        bad_buffer(grad_probs, (int64_t)d.T * d.K * 4, 4))
        return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    MoveArgs m = move_args(d, layout, grad_y, const_cast<uint16_t*>(expert_out), nullptr);
    return status_of(launch_probs_grad(m, grad_probs, static_cast<hipStream_t>(stream)));
}

int ep_indices_to_multihot(const ep_cfg_t* cfg, const int32_t* topk_ids, const float* probs,
                           uint8_t* routing_map, float* dense_probs, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if (grid_too_big(d, 64)) return EP_EINVAL;
    if (bad_buffer(topk_ids, (int64_t)d.T * d.K * 4, 4) || bad_buffer(routing_map, (int64_t)d.T * d.E, 1))
        return EP_EINVAL;
    if (dense_probs != nullptr && (bad_buffer(dense_probs, (int64_t)d.T * d.E * 4, 4) ||
                                   bad_buffer(probs, (int64_t)d.T * d.K * 4, 4)))
        return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    RouteArgs a;
    a.ids = const_cast<int32_t*>(topk_ids);
    a.probs = dense_probs != nullptr ? const_cast<float*>(probs) : nullptr;
    a.map = routing_map;
    a.dense_probs = dense_probs;
    a.flags = nullptr;
    a.T = d.T;
    a.K = d.K;
    a.E = d.E;
    return status_of(launch_indices_to_multihot(a, static_cast<hipStream_t>(stream)));
}

int ep_multihot_to_indices(const ep_cfg_t* cfg, const uint8_t* routing_map, const float* dense_probs,
                           int32_t* topk_ids, float* probs, int32_t* flags, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if (grid_too_big(d, 64)) return EP_EINVAL;
    if (bad_buffer(routing_map, (int64_t)d.T * d.E, 1) || bad_buffer(topk_ids, (int64_t)d.T * d.K * 4, 4))
        return EP_EINVAL;
    if (probs != nullptr && (bad_buffer(probs, (int64_t)d.T * d.K * 4, 4) ||
                             bad_buffer(dense_probs, (int64_t)d.T * d.E * 4, 4)))
        return EP_EINVAL;
    if (flags != nullptr && misaligned(flags, 4)) return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    RouteArgs a;
    a.ids = topk_ids;
    a.probs = probs;
    a.map = const_cast<uint8_t*>(routing_map);
    a.dense_probs = probs != nullptr ? const_cast<float*>(dense_probs) : nullptr;
    a.flags = flags;
    a.T = d.T;
    a.K = d.K;
    a.E = d.E;
    return status_of(launch_multihot_to_indices(a, static_cast<hipStream_t>(stream)));
}

int ep_route(const ep_cfg_t* cfg, const ep_route_t* route, const void* logits, const float* bias,
             const uint8_t* token_mask, int32_t* topk_ids, float* probs, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_route(d, route)) != EP_OK) return rc;
    if (grid_too_big(d, 64)) return EP_EINVAL;
    if (bad_buffer(logits, (int64_t)d.T * d.E * 2, 16) || misaligned(bias, 4) ||
        bad_buffer(topk_ids, (int64_t)d.T * d.K * 4, 4) || bad_buffer(probs, (int64_t)d.T * d.K * 4, 4))
        return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    TopkArgs a = topk_args(d, route, logits);
    a.bias = bias;
    a.mask = token_mask;
    a.ids = topk_ids;
    a.probs = probs;
    return status_of(launch_route(a, static_cast<hipStream_t>(stream)));
}

int ep_route_bwd(const ep_cfg_t* cfg, const ep_route_t* route, const void* logits, const int32_t* topk_ids,
                 const float* grad_probs, void* grad_logits, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_route(d, route)) != EP_OK) return rc;
    if (grid_too_big(d, 64)) return EP_EINVAL;
    if (bad_buffer(logits, (int64_t)d.T * d.E * 2, 16) || bad_buffer(grad_logits, (int64_t)d.T * d.E * 2, 16) ||
        bad_buffer(topk_ids, (int64_t)d.T * d.K * 4, 4) || bad_buffer(grad_probs, (int64_t)d.T * d.K * 4, 4))
        return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    TopkArgs a = topk_args(d, route, logits);
    a.ids = const_cast<int32_t*>(topk_ids);
    a.grad_probs = grad_probs;
    a.grad_logits = grad_logits;
    return status_of(launch_route_bwd(a, static_cast<hipStream_t>(stream)));
}

int ep_swiglu(const ep_cfg_t* cfg, const ep_layout_t* layout, int32_t inter, const uint16_t* h, const float* probs,
              uint16_t* act, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_rows(d)) != EP_OK) return rc;
    if (inter < 8 || inter > EP_MAX_EXPERT_DIM || inter % 8 != 0) return EP_EINVAL;
    if ((rc = check_layout_for_payload(d, layout)) != EP_OK) return rc;
    if (bad_buffer(h, d.R * inter * 4, 16) || bad_buffer(act, d.R * inter * 2, 16) || misaligned(probs, 4))
        return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    SwigluArgs a = {h, probs, nullptr, act, nullptr, layout->token_row, d.T, d.K, d.Kp, inter, d.R};
    if ((rc = status_of(launch_swiglu(a, st))) != EP_OK) return rc;
    return zero_pad(d, layout, act, (int64_t)inter * 2, st);
}

int ep_swiglu_bwd(const ep_cfg_t* cfg, const ep_layout_t* layout, int32_t inter, const uint16_t* h, const float* probs,
                  const uint16_t* grad_act, uint16_t* grad_h, float* grad_probs, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_rows(d)) != EP_OK) return rc;
    if (inter < 8 || inter > EP_MAX_EXPERT_DIM || inter % 8 != 0) return EP_EINVAL;
    if ((rc = check_layout_for_payload(d, layout)) != EP_OK) return rc;
    if (bad_buffer(h, d.R * inter * 4, 16) || bad_buffer(grad_act, d.R * inter * 2, 16) ||
        bad_buffer(grad_h, d.R * inter * 4, 16) || misaligned(probs, 4) || misaligned(grad_probs, 4))
        return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    SwigluArgs a = {h, probs, grad_act, grad_h, grad_probs, layout->token_row, d.T, d.K, d.Kp, inter, d.R};
    if ((rc = status_of(launch_swiglu_bwd(a, st))) != EP_OK) return rc;
    return zero_pad(d, layout, grad_h, (int64_t)inter * 4, st);
}

int ep_expert_gemm(const ep_cfg_t* cfg, const ep_layout_t* layout, int32_t in_dim, int32_t out_dim, const uint16_t* x,
                   const uint16_t* w, uint16_t* y, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_expert(d, layout, in_dim, out_dim, 8)) != EP_OK) return rc;
    if (bad_buffer(x, d.R * in_dim * 2, 16) || bad_buffer(w, 16, 16) || bad_buffer(y, d.R * out_dim * 2, 16))
        return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    ExpertArgs a = expert_args(d, layout, in_dim, out_dim, y);
    a.x = x;
    a.w = w;
    if ((rc = expert_status(launch_expert_gemm(a, st))) != EP_OK) return rc;
    return zero_pad(d, layout, y, (int64_t)out_dim * 2, st);
}

int ep_expert_gemm_bwd_x(const ep_cfg_t* cfg, const ep_layout_t* layout, int32_t in_dim, int32_t out_dim,
                         const uint16_t* grad_y, const uint16_t* w, uint16_t* grad_x, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_expert(d, layout, in_dim, out_dim, 8)) != EP_OK) return rc;
    if (bad_buffer(grad_y, d.R * out_dim * 2, 16) || bad_buffer(w, 16, 16) || bad_buffer(grad_x, d.R * in_dim * 2, 16))
        return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    ExpertArgs a = expert_args(d, layout, in_dim, out_dim, grad_x);
    a.gy = grad_y;
    a.w = w;
    if ((rc = expert_status(launch_expert_gemm_bwd_x(a, st))) != EP_OK) return rc;
    return zero_pad(d, layout, grad_x, (int64_t)in_dim * 2, st);
}

int ep_expert_gemm_bwd_w(const ep_cfg_t* cfg, const ep_layout_t* layout, int32_t in_dim, int32_t out_dim,
                         const uint16_t* grad_y, const uint16_t* x, void* grad_w, int32_t grad_type, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_expert(d, layout, in_dim, out_dim, 8)) != EP_OK) return rc;
    if (grad_type != EP_GRAD_BF16 && grad_type != EP_GRAD_F32 && grad_type != EP_GRAD_F32_ADD) return EP_EINVAL;
    if (bad_buffer(grad_y, d.R * out_dim * 2, 16) || bad_buffer(x, d.R * in_dim * 2, 16) || bad_buffer(grad_w, 16, 16))
        return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    ExpertArgs a = expert_args(d, layout, in_dim, out_dim, grad_w);
    a.gy = grad_y;
    a.x = x;
    a.grad_type = grad_type;
    return expert_status(launch_expert_gemm_bwd_w(a, static_cast<hipStream_t>(stream)));
}

int ep_expert_gemm_nvfp4(const ep_cfg_t* cfg, const ep_layout_t* layout, int32_t in_dim, int32_t out_dim,
                         const uint16_t* x, const uint8_t* codes, const uint8_t* scales, const uint16_t* rowscale,
                         uint16_t* y, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_expert(d, layout, in_dim, out_dim, 16)) != EP_OK) return rc;
    if (bad_buffer(x, d.R * in_dim * 2, 16) || bad_buffer(codes, 16, 16) || bad_buffer(scales, 16, 16) ||
        bad_buffer(rowscale, 8, 8) || bad_buffer(y, d.R * out_dim * 2, 16))
        return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    ExpertArgs a = expert_args(d, layout, in_dim, out_dim, y);
    a.x = x;
    a.codes = codes;
    a.scales = scales;
    a.rowscale = rowscale;
    if ((rc = expert_status(launch_expert_gemm_nvfp4(a, st))) != EP_OK) return rc;
    return zero_pad(d, layout, y, (int64_t)out_dim * 2, st);
}

int ep_lora_down(const ep_cfg_t* cfg, const ep_layout_t* layout, const ep_lora_t* lora, int32_t in_dim,
                 const uint16_t* x, float* u, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_block(d, layout, in_dim, 8, 8)) != EP_OK) return rc;
    if ((rc = check_lora(d, lora, true, false)) != EP_OK) return rc;
    if (bad_buffer(x, d.R * in_dim * 2, 16) || bad_buffer(u, d.R * lora->rank * 4, 16)) return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    BlockArgs a = block_args(d, layout, lora, in_dim, 8, nullptr, nullptr);
    a.e.x = x;
    if ((rc = expert_status(launch_lora_down(a, u, st))) != EP_OK) return rc;
    return zero_pad(d, layout, u, (int64_t)lora->rank * 4, st);
}

int ep_lora_bwd_u(const ep_cfg_t* cfg, const ep_layout_t* layout, const ep_lora_t* lora, int32_t out_dim,
                  const uint16_t* grad_y, float* grad_u, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_block(d, layout, 8, out_dim, 8)) != EP_OK) return rc;
    if ((rc = check_lora(d, lora, false, true)) != EP_OK) return rc;
    if (bad_buffer(grad_y, d.R * out_dim * 2, 16) || bad_buffer(grad_u, d.R * lora->rank * 4, 16)) return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    BlockArgs a = block_args(d, layout, lora, 8, out_dim, nullptr, nullptr);
    a.e.gy = grad_y;
    if ((rc = expert_status(launch_lora_bwd_u(a, grad_u, st))) != EP_OK) return rc;
    return zero_pad(d, layout, grad_u, (int64_t)lora->rank * 4, st);
}

int ep_expert_gemm_lora(const ep_cfg_t* cfg, const ep_layout_t* layout, const ep_lora_t* lora, int32_t in_dim,
                        int32_t out_dim, const uint16_t* x, const uint16_t* w, const float* u, uint16_t* y, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_block(d, layout, in_dim, out_dim, 8)) != EP_OK) return rc;
    if ((rc = check_lora(d, lora, false, true)) != EP_OK) return rc;
    if (bad_buffer(x, d.R * in_dim * 2, 16) || bad_buffer(w, 16, 16) || bad_buffer(u, d.R * lora->rank * 4, 16) ||
        bad_buffer(y, d.R * out_dim * 2, 16))
        return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    BlockArgs a = block_args(d, layout, lora, in_dim, out_dim, u, y);
    a.e.x = x;
    a.e.w = w;
    if ((rc = expert_status(launch_gemm_lora(a, st))) != EP_OK) return rc;
    return zero_pad(d, layout, y, (int64_t)out_dim * 2, st);
}

int ep_expert_gemm_nvfp4_lora(const ep_cfg_t* cfg, const ep_layout_t* layout, const ep_lora_t* lora, int32_t in_dim,
                              int32_t out_dim, const uint16_t* x, const uint8_t* codes, const uint8_t* scales,
                              const uint16_t* rowscale, const float* u, uint16_t* y, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_block(d, layout, in_dim, out_dim, 16)) != EP_OK) return rc;
    if ((rc = check_lora(d, lora, false, true)) != EP_OK) return rc;
    if (bad_buffer(x, d.R * in_dim * 2, 16) || bad_buffer(codes, 16, 16) || bad_buffer(scales, 16, 16) ||
        bad_buffer(rowscale, 8, 8) || bad_buffer(u, d.R * lora->rank * 4, 16) || bad_buffer(y, d.R * out_dim * 2, 16))
        return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    BlockArgs a = block_args(d, layout, lora, in_dim, out_dim, u, y);
    a.e.x = x;
    a.e.codes = codes;
    a.e.scales = scales;
    a.e.rowscale = rowscale;
    if ((rc = expert_status(launch_gemm_nvfp4_lora(a, st))) != EP_OK) return rc;
    return zero_pad(d, layout, y, (int64_t)out_dim * 2, st);
}

int ep_expert_gemm_bwd_x_lora(const ep_cfg_t* cfg, const ep_layout_t* layout, const ep_lora_t* lora, int32_t in_dim,
                              int32_t out_dim, const uint16_t* grad_y, const uint16_t* w, const float* grad_u,
                              uint16_t* grad_x, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_block(d, layout, in_dim, out_dim, 8)) != EP_OK) return rc;
    if ((rc = check_lora(d, lora, true, false)) != EP_OK) return rc;
    if (bad_buffer(grad_y, d.R * out_dim * 2, 16) || bad_buffer(w, 16, 16) ||
        bad_buffer(grad_u, d.R * lora->rank * 4, 16) || bad_buffer(grad_x, d.R * in_dim * 2, 16))
        return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    BlockArgs a = block_args(d, layout, lora, in_dim, out_dim, grad_u, grad_x);
    a.e.gy = grad_y;
    a.e.w = w;
    if ((rc = expert_status(launch_gemm_bwd_x_lora(a, st))) != EP_OK) return rc;
    return zero_pad(d, layout, grad_x, (int64_t)in_dim * 2, st);
}

int ep_lora_bwd_w(const ep_cfg_t* cfg, const ep_layout_t* layout, const ep_lora_t* lora, int32_t in_dim,
                  int32_t out_dim, const uint16_t* x, const uint16_t* grad_y, const float* u, const float* grad_u,
                  void* grad_a, void* grad_b, int32_t grad_type, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_block(d, layout, in_dim, out_dim, 8)) != EP_OK) return rc;
    if ((rc = check_lora(d, lora, false, false)) != EP_OK) return rc;
    if (grad_type != EP_GRAD_BF16 && grad_type != EP_GRAD_F32 && grad_type != EP_GRAD_F32_ADD) return EP_EINVAL;
    if (bad_buffer(x, d.R * in_dim * 2, 16) || bad_buffer(grad_y, d.R * out_dim * 2, 16) ||
        bad_buffer(u, d.R * lora->rank * 4, 16) || bad_buffer(grad_u, d.R * lora->rank * 4, 16) ||
        bad_buffer(grad_a, 16, 16) || bad_buffer(grad_b, 16, 16))
        return EP_EINVAL;
    BlockArgs a = block_args(d, layout, lora, in_dim, out_dim, u, nullptr);
    if ((rc = expert_status(check_lora_bwd_w(a))) != EP_OK) return rc;
    if ((rc = check_device()) != EP_OK) return rc;
    a.e.x = x;
    a.e.gy = grad_y;
    a.e.grad_type = grad_type;
    return expert_status(launch_lora_bwd_w(a, grad_u, grad_a, grad_b,
                                           static_cast<hipStream_t>(stream)));
}

int ep_expert_gated(const ep_cfg_t* cfg, const ep_layout_t* layout, const ep_lora_t* lora, int32_t in_dim, int32_t inter,
                    const uint16_t* x, const uint16_t* w, const float* probs, const float* ulora, uint16_t* act,
                    void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_gated(d, layout, lora, in_dim, inter, 8, ulora, probs)) != EP_OK) return rc;
    if (bad_buffer(x, d.R * in_dim * 2, 16) || bad_buffer(w, 16, 16) || bad_buffer(act, d.R * inter * 2, 16))
        return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    BlockArgs a = gated_args(d, layout, lora, in_dim, inter, ulora, probs, act);
    a.e.x = x;
    a.e.w = w;
    if ((rc = expert_status(launch_gated(a, st))) != EP_OK) return rc;
    return zero_pad(d, layout, act, (int64_t)inter * 2, st);
}

int ep_expert_gated_nvfp4(const ep_cfg_t* cfg, const ep_layout_t* layout, const ep_lora_t* lora, int32_t in_dim,
                          int32_t inter, const uint16_t* x, const uint8_t* codes, const uint8_t* scales,
                          const uint16_t* rowscale, const float* probs, const float* ulora, uint16_t* act, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_gated(d, layout, lora, in_dim, inter, 16, ulora, probs)) != EP_OK) return rc;
    if ((int64_t)inter * in_dim >= int64_t(1) << 34) return EP_EINVAL;  // an expert's scales are reached by 32-bit offsets
    if (bad_buffer(x, d.R * in_dim * 2, 16) || bad_buffer(codes, 16, 16) || bad_buffer(scales, 16, 16) ||
        bad_buffer(rowscale, 8, 8) || bad_buffer(act, d.R * inter * 2, 16))
        return EP_EINVAL;
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    BlockArgs a = gated_args(d, layout, lora, in_dim, inter, ulora, probs, act);
    a.e.x = x;
    a.e.codes = codes;
    a.e.scales = scales;
    a.e.rowscale = rowscale;
    if ((rc = expert_status(launch_gated_nvfp4(a, st))) != EP_OK) return rc;
    return zero_pad(d, layout, act, (int64_t)inter * 2, st);
}

int ep_expert_gated_bwd(const ep_cfg_t* cfg, const ep_layout_t* layout, const ep_lora_t* lora, int32_t in_dim,
                        int32_t inter, const uint16_t* x, const uint16_t* w, const float* probs, const float* ulora,
                        const uint16_t* grad_act, uint16_t* grad_h, uint16_t* act, float* grad_probs, void* workspace,
                        int64_t workspace_bytes, void* stream) {
    Shape d;
    int rc = derive(cfg, &d);
    if (rc != EP_OK) return rc;
    if ((rc = check_gated(d, layout, lora, in_dim, inter, 8, ulora, probs)) != EP_OK) return rc;
    if (bad_buffer(x, d.R * in_dim * 2, 16) || bad_buffer(w, 16, 16) || bad_buffer(grad_act, d.R * inter * 2, 16) ||
        bad_buffer(grad_h, d.R * inter * 4, 16) || misaligned(act, 16))
        return EP_EINVAL;
    if (grad_probs != nullptr) {
        const int64_t need = (int64_t)d.T * d.K * ((inter + EP_GATED_PART - 1) / EP_GATED_PART) * 4;
        if (misaligned(grad_probs, 4) || workspace_bytes < need || bad_buffer(workspace, need, 16)) return EP_EINVAL;
        if (bad_buffer(layout->token_row, (int64_t)d.T * d.Kp * 4, 4)) return EP_EINVAL;
    }
    if ((rc = check_device()) != EP_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    BlockArgs a = gated_args(d, layout, lora, in_dim, inter, ulora, probs, act);
    a.e.x = x;
    a.e.w = w;
    a.grad_act = grad_act;
    a.grad_h = grad_h;
    a.grad_probs = grad_probs;
    a.parts = grad_probs != nullptr ? static_cast<float*>(workspace) : nullptr;
    if ((rc = expert_status(launch_gated_bwd(a, st))) != EP_OK) return rc;
    if (act != nullptr && (rc = zero_pad(d, layout, act, (int64_t)inter * 2, st)) != EP_OK) return rc;
    return zero_pad(d, layout, grad_h, (int64_t)inter * 4, st);
}

}  // extern "C"
