"""The feed-forward block at sizes for each way of cutting its three products, those with tiles
of 192 rows among them."""

import pytest
import torch

import test_gpu_ffn as base

pytestmark = pytest.mark.gpu

BF, F16 = torch.bfloat16, torch.float16

# rows by H by I; first product, second product, dh
SIZES = [(2990, 1152, 1856),    # 192 x 256, 128 x 128, 192 x 128
         (4694, 160, 800),      # 192 x 256, 64 x 64, 192 x 128
         (576, 5984, 4672),     # 192 x 128, 128 x 128 both
         (8331, 544, 192),      # 128 x 128, 192 x 128, 128 x 128
         (1931, 5184, 416),     # 64 x 128, 192 x 256, 128 x 128 in parts
         (2679, 928, 3168),     # 256 x 256 with quarters left over, 128 x 128, 192 x 256
         (1456, 4544, 128),     # 64 x 128 in parts, 128 x 256, 64 x 64 in parts
         (4373, 96, 1760),      # 256 x 256, 64 x 64, 128 x 256
         (770, 512, 4096),      # 128 x 256, 64 x 128 in parts, 128 x 128
         (3804, 4768, 160),     # 64 x 128, 256 x 256 with quarters, 128 x 128 in parts
         (8677, 4576, 160),     # 128 x 128, 256 x 256 with halves, 128 x 128
         (8986, 224, 4288),     # 256 x 256, 128 x 128, 256 x 256 with halves
         (13689, 672, 832),     # 256 x 256 with halves, 192 x 256, 256 x 256
         (11650, 128, 1472),    # 256 x 256 with quarters, 64 x 128, 256 x 256 with quarters
         (7135, 2208, 768),     # 192 x 256, 256 x 256, 192 x 128
         (245, 512, 2880)]      # 64 x 128, 64 x 64 in parts, 64 x 64


@pytest.mark.parametrize("T,H,I", SIZES)
def test_forward_whole_numbers(T, H, I):
    base.test_forward_whole_numbers(T, H, I, F16 if T % 2 else BF)


@pytest.mark.parametrize("T,H,I", SIZES)
def test_backward_whole_numbers(T, H, I):
    base.test_backward_whole_numbers(T, H, I, BF if T % 2 else F16)


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("T,H,I", [(2990, 1152, 1856), (2679, 928, 3168), (1931, 2080, 416)])
def test_normal_values(T, H, I, dt):
    base.test_normal_values(T, H, I, 2.0, dt)
