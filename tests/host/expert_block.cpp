// The launches of one of the experts' sources (SOURCE, a number: which one) over
// layouts and sizes where operands and tiles end, on the host.  Every operand ends with
// its allocation.  Each case runs with loads to LDS that land at once and as late as the
// waits allow, each with either of a workgroup's ends ahead: the results have to be the
// same bits.
#include <hip/hip_runtime.h>

#if SOURCE == 0
#include "expert_gated.hip"
#elif SOURCE == 1
#include "expert_lora.hip"
#elif SOURCE == 2
#include "expert_nvfp4_block.hip"
#elif SOURCE == 3
#include "expert_gemm.hip"
#else
#include "expert_nvfp4.hip"
#endif

using namespace epx;

namespace {

uint32_t seed = 1;
uint32_t random_bits() {
    seed = seed * 1664525u + 1013904223u;
    return seed >> 8 ^ seed << 13;
}

template <typename T>
T* array(size_t n) {
    return static_cast<T*>(host::alloc(n * sizeof(T)));
}

// bf16 values of magnitude below 2
uint16_t* values(size_t n) {
    uint16_t* const p = array<uint16_t>(n);
    for (size_t k = 0; k < n; ++k) p[k] = (uint16_t)(random_bits() & 0xBFFF);
    return p;
}

// Values of which some are infinite.
uint16_t* wild_values(size_t n) {
    uint16_t* const p = values(n);
    for (size_t k = random_bits() % 97; k < n; k += 97) p[k] = 0x7F80;
    return p;
}

uint8_t* bytes(size_t n) {
    uint8_t* const p = array<uint8_t>(n);
    for (size_t k = 0; k < n; ++k) p[k] = (uint8_t)(random_bits() >> 3);
    return p;
}

float* floats(size_t n) {
    float* const p = array<float>(n);
    for (size_t k = 0; k < n; ++k) p[k] = (float)(random_bits() % 1000) / 999.0f;
    return p;
}

// One segment's experts (the first group's last where one is shared), a token a row.
struct Layout {
    BlockArgs a;
    std::vector<int32_t> rows;

    Layout(const std::vector<int32_t>& counts, bool shared, int32_t in, int32_t on, int32_t rank, int32_t adapters)
        : a{}, rows(counts) {
        const int32_t G = (int32_t)counts.size();
        int32_t R = 0;
        int32_t* const c = array<int32_t>(G);
        int32_t* const offsets = array<int32_t>(G + 1);
        int32_t* const base = array<int32_t>(2);
        for (int32_t g = 0; g < G; ++g) {
            c[g] = counts[g];
            offsets[g] = R;
            R += counts[g];
        }
        offsets[G] = base[1] = R;
        base[0] = 0;
        ExpertArgs& e = a.e;
        e.counts = c;
        e.row_offsets = offsets;
        e.seg_base = base;
        e.in = in;
        e.on = on;
        e.E = e.E_loc = G - shared;
        e.S = 1;
        e.G = e.NG = G;
        e.shared = shared;
        e.R = R;
        e.slots = R;
        a.T = R;
        a.K = a.Kp = 1;
        int32_t* const src = array<int32_t>(2 * R);
        int32_t* const token_row = array<int32_t>(R);
        for (int32_t r = 0; r < R; ++r) {
            src[2 * r] = token_row[r] = R - 1 - r;
            src[2 * r + 1] = 0;
        }
        a.src_info = src;
        a.token_row = token_row;
        if (rank > 0) {
            int32_t* const of = array<int32_t>(R);
            for (int32_t t = 0; t < R; ++t) of[t] = (int32_t)(random_bits() % (uint32_t)(adapters + 1)) - 1;
            a.l = {of, nullptr, nullptr, floats(adapters), adapters, rank};
        }
    }
    int64_t R() const { return a.e.R; }
    int64_t experts() const { return (int64_t)rows.size(); }
};

struct Output {
    void* at;
    size_t bytes;
};

// Runs call four times and compares the outputs.
template <typename Call>
void compare(const std::vector<Output>& outputs, Call call) {
    std::vector<std::vector<char>> want;
    for (int k = 0; k < 4; ++k) {
        host::late = k % 2;
        host::backwards = k / 2;
        for (const Output& o : outputs) memset(o.at, 0x7A, o.bytes);
        if (call() != hipSuccess) host::fail("the launch is refused");
        for (size_t n = 0; n < outputs.size(); ++n) {
            const char* const p = static_cast<const char*>(outputs[n].at);
            if (k == 0)
                want.emplace_back(p, p + outputs[n].bytes);
            else if (memcmp(want[n].data(), p, outputs[n].bytes) != 0)
                host::fail("output %zu depends on when loads land and which wave is ahead (%s loads, the %s wave first)", n,
                           host::late ? "late" : "early", host::backwards ? "last" : "first");
        }
    }
}

const std::vector<std::vector<int32_t>> kLayouts = {
    {1},                        // a single row
    {5, 0, 17},                 // few rows
    {21, 30, 19},               // up to 32
    {57, 0, 40, 33},            // up to 64
    {130, 20, 100},             // every kind of tile but the tallest
    {0, 300, 1, 200, 128, 33},  // all kinds
    {1060, 20, 900, 100},       // full tiles and what is left over, tiles of one height
};

std::string name(const char* kernel, const std::vector<int32_t>& rows, int32_t in, int32_t out, int32_t rank) {
    std::string s = std::string(kernel) + " in=" + std::to_string(in) + " out=" + std::to_string(out) + " rank=" + std::to_string(rank) + " rows=";
    for (int32_t r : rows) s += std::to_string(r) + " ";
    return s;
}

void one(const std::vector<int32_t>& rows, bool shared, int32_t in, int32_t out, int32_t rank) {
    // out: columns of act where gated, of the product where not
    const int32_t adapters = 3;
#if SOURCE == 0
    Layout l(rows, shared, in, 2 * out, rank, adapters);
    BlockArgs& a = l.a;
    a.I = out;
    a.e.x = values(l.R() * in);
    a.e.w = values(l.experts() * 2 * out * in);
    if (rank > 0) {
        a.l.b = (rank == 40 ? wild_values : values)(l.experts() * adapters * 2 * out * rank);
        a.u = floats(l.R() * rank);
    }
    a.probs = floats(l.R());
    a.e.out = array<uint16_t>(l.R() * out);
    host::what = name("gated", rows, in, out, rank);
    compare({{a.e.out, (size_t)l.R() * out * 2}}, [&] { return launch_gated(a, nullptr); });
    a.grad_act = values(l.R() * out);
    a.grad_h = array<uint16_t>(l.R() * 2 * out);
    a.grad_probs = array<float>(l.R());
    const size_t parts = l.R() * ((out + kGatedPart - 1) / kGatedPart);
    a.parts = array<float>(parts);
    host::what = name("gated_bwd", rows, in, out, rank);
    compare({{a.e.out, (size_t)l.R() * out * 2}, {a.grad_h, (size_t)l.R() * out * 4}, {a.grad_probs, (size_t)l.R() * 4}, {a.parts, parts * 4}},
            [&] { return launch_gated_bwd(a, nullptr); });
#elif SOURCE == 1
    if (rank == 0) return;
    Layout l(rows, shared, in, out, rank, adapters);
    BlockArgs& a = l.a;
    a.e.x = values(l.R() * in);
    a.e.gy = values(l.R() * out);
    a.e.w = values(l.experts() * out * in);
    a.l.a = (rank == 40 ? wild_values : values)(l.experts() * adapters * rank * in);
    a.l.b = (rank == 40 ? wild_values : values)(l.experts() * adapters * out * rank);
    float *const u = array<float>(l.R() * rank), *const gu = array<float>(l.R() * rank);
    const size_t u_bytes = (size_t)l.R() * rank * 4;
    host::what = name("lora_down", rows, in, out, rank);
    compare({{u, u_bytes}}, [&] { return launch_lora_down(a, u, nullptr); });
    host::what = name("lora_bwd_u", rows, in, out, rank);
    compare({{gu, u_bytes}}, [&] { return launch_lora_bwd_u(a, gu, nullptr); });
    a.e.slots = 64 * kCus;  // as a layout of many slots of which few have rows: tiles of 64
    host::what = name("lora_down of 64", rows, in, out, rank);
    compare({{u, u_bytes}}, [&] { return launch_lora_down(a, u, nullptr); });
    host::what = name("lora_bwd_u of 64", rows, in, out, rank);
    compare({{gu, u_bytes}}, [&] { return launch_lora_bwd_u(a, gu, nullptr); });
    a.e.slots = l.R();
    a.u = u;
    a.e.out = array<uint16_t>(l.R() * out);
    host::what = name("gemm_lora", rows, in, out, rank);
    compare({{a.e.out, (size_t)l.R() * out * 2}}, [&] { return launch_gemm_lora(a, nullptr); });
    a.e.out = array<uint16_t>(l.R() * in);
    a.u = gu;
    host::what = name("gemm_bwd_x_lora", rows, in, out, rank);
    compare({{a.e.out, (size_t)l.R() * in * 2}}, [&] { return launch_gemm_bwd_x_lora(a, nullptr); });
    a.u = u;
    const size_t na = l.experts() * adapters * rank * in, nb = l.experts() * adapters * out * rank;
    for (int type : {EP_GRAD_BF16, EP_GRAD_F32}) {
        a.e.grad_type = type;
        const size_t each = type == EP_GRAD_BF16 ? 2 : 4;
        void *const ga = host::alloc(na * each), *const gb = host::alloc(nb * each);
        host::what = name("lora_bwd_w", rows, in, out, rank);
        compare({{ga, na * each}, {gb, nb * each}}, [&] { return launch_lora_bwd_w(a, gu, ga, gb, nullptr); });
    }
#elif SOURCE == 3
    if (rank != 0) return;
    Layout l(rows, shared, in, out, 0, 0);
    ExpertArgs& a = l.a.e;
    const size_t nx = l.R() * in, ny = l.R() * out, nw = l.experts() * out * in;
    a.x = values(nx);
    a.gy = values(ny);
    a.w = values(nw);
    a.out = array<uint16_t>(ny);
    for (int64_t slots : {l.R(), int64_t(1) << 16}) {  // by which the tiles' sizes are chosen
        a.slots = slots;
        a.out = array<uint16_t>(ny);
        host::what = name("gemm", rows, in, out, rank);
        compare({{a.out, ny * 2}}, [&] { return launch_expert_gemm(a, nullptr); });
        a.out = array<uint16_t>(nx);
        host::what = name("gemm_bwd_x", rows, in, out, rank);
        compare({{a.out, nx * 2}}, [&] { return launch_expert_gemm_bwd_x(a, nullptr); });
        a.out = array<uint16_t>(nw);
        host::what = name("gemm_bwd_w", rows, in, out, rank);
        compare({{a.out, nw * 2}}, [&] { return launch_expert_gemm_bwd_w(a, nullptr); });
    }
#elif SOURCE == 4
    if (rank != 0) return;
    Layout l(rows, shared, in, out, 0, 0);
    ExpertArgs& a = l.a.e;
    a.x = values(l.R() * in);
    a.codes = bytes(l.experts() * out * in / 2);
    a.scales = bytes(l.experts() * out * in / 16);
    a.rowscale = values(l.experts() * out);
    a.out = array<uint16_t>(l.R() * out);
    host::what = name("gemm_nvfp4", rows, in, out, rank);
    compare({{a.out, (size_t)l.R() * out * 2}}, [&] { return launch_expert_gemm_nvfp4(a, nullptr); });
#else
    for (bool gated : {true, false}) {
        if (!gated && rank == 0) continue;
        const int32_t on = gated ? 2 * out : out;
        Layout l(rows, shared, in, on, rank, adapters);
        BlockArgs& a = l.a;
        a.I = out;
        a.e.x = values(l.R() * in);
        a.e.codes = bytes(l.experts() * on * in / 2);
        a.e.scales = bytes(l.experts() * on * in / 16);
        a.e.rowscale = values(l.experts() * on);
        if (rank > 0) {
            a.l.b = (rank == 40 ? wild_values : values)(l.experts() * adapters * on * rank);
            a.u = floats(l.R() * rank);
        }
        a.probs = floats(l.R());
        a.e.out = array<uint16_t>(l.R() * out);
        host::what = name(gated ? "gated_nvfp4" : "gemm_nvfp4_lora", rows, in, out, rank);
        compare({{a.e.out, (size_t)l.R() * out * 2}}, [&] { return gated ? launch_gated_nvfp4(a, nullptr) : launch_gemm_nvfp4_lora(a, nullptr); });
    }
#endif
}

}  // namespace

// Arguments: the in_dims, "x", the widths.
int main(int argc, char** argv) {
    host::start();
    std::vector<int32_t> ins, outs;
    int k = 1;
    for (; k < argc && strcmp(argv[k], "x") != 0; ++k) ins.push_back(atoi(argv[k]));
    for (++k; k < argc; ++k) outs.push_back(atoi(argv[k]));
    int cases = 0;
    for (int32_t in : ins)
        for (int32_t out : outs)
            for (size_t n = 0; n < kLayouts.size(); ++n)
                for (int32_t rank : {0, 40}) {
                    one(kLayouts[n], n % 2 == 1, in, out, rank);
                    host::free_all();
                    ++cases;
                }
    printf("%d cases\n", cases);
    return 0;
}
