// Which kernels calls of the feed-forward operators take, from the library's own plan:
//
//   ff_plan < calls        each line "f32|bf16 linear|gated none|relu|silu|gelu rows C N": its kernels, one line a call
//   ff_plan sweep COUNT MOST   the kernels that COUNT calls of many sizes take, up to MOST multiplications in one
//                              product, each with the call of the fewest
//
// Operands are contiguous and aligned.  A kernel is "type product tile how": product y, gated, grad_x or grad_w
// (with " terms" where the gradient of z has two, and " again" where the backward makes z); tile its columns and
// rows of the result, "any" through registers, "chunked" or "rows" (sixteens of rows) for few rows; how "whole",
// "pieces" or both.  Pieces are joined by 1 to 32 lanes, the backward of few channels is "small".
#include <cmath>
#include <cstdio>
#include <cstring>
#include <map>
#include <random>
#include <string>
#include <vector>

#include "ff_plan.hpp"

using namespace ddpm::ff;

struct Call {
    bool bf16, gated;
    int act;
    int64_t rows, C, N;
    double work() const { return (double)rows * C * N * (gated ? 2 : 1); }
};
static const char *const kActs[] = {"none", "relu", "silu", "gelu"};

static void product(std::vector<std::string> &k, const Call &c, Kind kind, const char *name, int64_t np, int64_t nq, int64_t nk, int terms, bool direct) {
    const std::string head = std::string(c.bf16 ? "bf16 " : "f32 ") + name + (terms == 2 ? " terms" : "") + " ";
    if (few_rows(kind, np, nq, nk, c.bf16, direct)) {
        k.push_back(head + (direct ? "chunked " : "rows ") + std::to_string((nq + 15) / 16));
        return;
    }
    const Cut cut = cut_of(kind, np, nq, nk, terms, c.bf16, direct);
    const Form f = form_of(c.bf16, kind, cut.form);
    k.push_back(head + (direct ? std::to_string(f.kp()) + "x" + std::to_string(f.kq()) : "any") +
                (cut.pieces == 1 ? " whole" : cut.whole ? " both" : " pieces"));
    if (cut.pieces > 1) k.push_back(head + "joined by " + std::to_string(finish_lanes(cut.pieces)));
}

static std::vector<std::string> kernels(const Call &c) {
    const Sizes s = {c.rows, c.C, c.N, c.gated ? 2 * c.N : c.N};
    const Kind kind = c.gated ? kGatedForward : kForward;
    const char *name = c.gated ? "gated" : "y";
    const bool through = c.gated || c.act != DDPM_ACT_NONE, whole_c = c.C % chunk(c.bf16) == 0;
    std::vector<std::string> k;
    product(k, c, kind, name, s.N, s.rows, s.C, 1, whole_c || forward_copies(kind, s, c.bf16));
    const Room r = backward_room(kind, s, through, c.act, c.bf16);
    if (r.small) {
        k.push_back(std::string(c.bf16 ? "bf16" : "f32") + (c.gated ? " gated" : "") + " small");
        return k;
    }
    const int terms = two_terms(kind, through, c.act, c.bf16) ? 2 : 1;
    const bool x = whole_c || r.copies, dz = r.own_dz || c.N % chunk(c.bf16) == 0;
    if (r.again) product(k, c, kind, (std::string(name) + " again").c_str(), s.N, s.rows, s.C, 1, x);
    product(k, c, kGradX, "grad_x", s.C, s.rows, s.width, terms, x && dz);
    product(k, c, kGradWeight, "grad_w", s.C, s.width, s.rows, terms, x && dz);
    return k;
}

int main(int argc, char **argv) {
    if (argc == 4 && !std::strcmp(argv[1], "sweep")) {
        std::map<std::string, Call> found;
        std::mt19937_64 rng(1);
        const auto size = [&](double lo, double hi) {
            const int64_t v = std::llround(std::exp(std::uniform_real_distribution<>(std::log(lo), std::log(hi))(rng)));
            return rng() % 2 ? v : (v + 7) / 8 * 8;
        };
        for (long n = std::atol(argv[2]); n > 0; --n) {
            const Call c = {rng() % 2 == 0, rng() % 2 == 0, (int)(rng() % 3), size(1, 70000), size(1, 9000), size(1, 9000)};
            if (c.work() > std::atof(argv[3])) continue;
            for (const std::string &k : kernels(c)) {
                const auto at = found.find(k);
                if (at == found.end() || c.work() < at->second.work()) found[k] = c;
            }
        }
        for (const auto &[k, c] : found)
            std::printf("%s\t%s %s %s %lld %lld %lld\n", k.c_str(), c.bf16 ? "bf16" : "f32", c.gated ? "gated" : "linear", kActs[c.act],
                        (long long)c.rows, (long long)c.C, (long long)c.N);
        return 0;
    }
    char type[8], op[8], act[8];
    long long rows, C, N;
    while (std::scanf("%7s %7s %7s %lld %lld %lld", type, op, act, &rows, &C, &N) == 6) {
        Call c = {!std::strcmp(type, "bf16"), !std::strcmp(op, "gated"), 0, rows, C, N};
        while (c.act < 3 && std::strcmp(act, kActs[c.act])) ++c.act;
        for (const std::string &k : kernels(c)) std::printf("%s;", k.c_str());
        std::printf("\n");
    }
    return 0;
}
