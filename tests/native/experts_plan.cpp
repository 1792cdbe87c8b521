// The kernels that calls of skinny_experts take (csrc/experts_plan.hpp): for every line of standard
// input, "type M E k H", those of its first pass; with the argument "all", every kernel that
// calls choose among.
#include <cstdio>
#include <cstring>

#include "../../bf16_skinny_gemm_amd/csrc/experts_plan.hpp"

using namespace skg_host;

namespace {

void say_up(int type, bool wave, const UpPlan &u)
{
    std::printf("up %d %d %d %d %d %d\n", type, wave, u.rows, u.waves, u.ring, u.room);
}

void say_down(int type, const DownPlan &d) { std::printf("down %d %d %d %d %d\n", type, d.rows, d.waves, d.ring, d.tokens); }

}  // namespace

int main(int argc, char **argv)
{
    if (argc > 1 && !std::strcmp(argv[1], "all")) {
        for (int type = SKINNY_WEIGHTS_BF16; type <= SKINNY_WEIGHTS_INT8_ROW; ++type)
            for (int rows : {4, 8, 16, 32}) {
                for (int wave = 0; wave < 2; ++wave) {
                    if (resident_offered(type, rows, wave))
                        for (int ring : kResidentRings)
                            say_up(type, wave, up_resident(type, rows, wave, ring));
                    say_up(type, wave, up_streamed(type, rows, wave));
                }
                for (int tokens : {16, 64, 128})
                    if (rows < 32 || tokens > 16)
                        say_down(type, down_of(type, rows, tokens));
            }
        return 0;
    }
    int type, M, E, k, H;
    while (std::scanf("%d %d %d %d %d", &type, &M, &E, &k, &H) == 5) {
        const bool wave = M * k <= kWavePairs;
        const UpPlan u = up_plan(type, tile_rows(type, M, E, k, H), wave, H);
        std::printf("%d ", u.rows);
        say_up(type, wave, u);
        std::printf("%d ", u.rows);
        say_down(type, down_of(type, u.rows, tokens_room(M)));
    }
    return 0;
}
