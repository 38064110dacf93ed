// attend_constants.cpp -- the constants with which the paged cache's kernels
// divide an attention call (few rows, few rows of an 8-bit cache, many rows), for
// the tests of the division.
#include "../tenant_lora_serving_amd/csrc/attend_kernels.h"

extern "C" void attend_constants(int kind, int *to) {
    const bool many = kind == 2;
    to[0] = many ? st::kManyRows : st::kFewRows;
    to[1] = many ? st::kManyFixed : kind == 1 ? st::kFewFixed8 : st::kFewFixed;
    to[2] = many ? st::kManyLeast : st::kFewLeast;
    to[3] = many ? st::kManyWhole : st::kFewWhole;
    to[4] = many ? st::kManyStep : st::kFewStep;
    to[5] = many ? st::kManyGroups : st::kFewGroups;
}
